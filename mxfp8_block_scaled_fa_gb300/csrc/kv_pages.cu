// kv_pages.cu -- pages of the 4-bit cache that several requests share: forking a request's
// pages, copying blocks, and giving pages back to the ring of free blocks.
//
// refs[b] counts the owners of block b beside the first: kv_plan's blocks have 0.
//   fork   request d gets the first c tokens of request s: each whole page has one owner more; a last page
//          that is not full is written again by both, so d gets a new block for it (the k-th such fork the
//          k-th free block) and the pair (old, new) is a block to copy, layer by layer.  Entries that s has given up
//          are not shared
//   free   each page given up has one owner fewer; blocks without an owner go to the ring, in ascending order
// Counts change by whole-number atomics, so no result depends on timing: which of a block's owners comes last
// is not seen, as blocks are collected by looking at the counts afterwards.
#include <cooperative_groups.h>

#include "kv_fp4.cuh"
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

namespace mxfa {

static __device__ unsigned g_status_kv_pages;

namespace {

constexpr int kThreads = 256;
constexpr int kForkThreads = 512;
constexpr int kCopyThreads = 512;
constexpr int kSegment = 2048;  // table entries of a CTA
constexpr int kScan = 1024;     // threads of a CTA that collects
constexpr int kCluster = 8;
// Table entries, at most, that the collecting cluster gives up itself: on the GPU 64 x 63 entries take 6.5 us with a
// kernel of their own and 6.9 without, 64 x 250 entries 7.8 and 9.7; the launch costs the host 3 us more.
constexpr int64_t kInside = 4096;

struct Fork {
  int src, dst, len, whole;  // whole pages
  int gap, gap_end;          // entries gap .. gap_end - 1 were given up
};
__device__ __forceinline__ bool fork_of(const KvForkArgs& a, int f, Fork& x) {
  x.src = __ldg(a.src + f), x.dst = __ldg(a.dst + f), x.len = __ldg(a.lens + f);
  x.gap = a.gap_first ? __ldg(a.gap_first + f) : 0;
  x.gap_end = a.gap_first ? __ldg(a.gap_end + f) : 0;
  if (x.src < 0 || x.src >= a.R || x.dst < 0 || x.dst >= a.R || x.src == x.dst) return false;
  if (x.len < 0 || x.len > int64_t(a.width) << a.page_shift) return false;
  x.whole = x.len >> a.page_shift;
  return x.gap >= 0 && x.gap_end >= x.gap && x.gap_end <= x.whole;
}

__device__ __forceinline__ int64_t in_ring(int64_t i, int64_t size) { return (i % size + size) % size; }

// The last pages of all forks that are not full, and the ring: one CTA, so that a fork's place in the ring is a sum over
// those before it, each looked at once, and the ring's counters may be written over.  N forks of a thread one behind another.
template <int N>
__device__ __forceinline__ void fork_parts(const KvForkArgs& a) {
  __shared__ int s_sum[kForkThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t head = a.ring_in[0], tail = a.ring_in[1];
  const int64_t room = tail - head;
  const int64_t avail = room < 0 ? 0 : room < a.ring_size ? room : a.ring_size;
  const int64_t first = in_ring(head, a.ring_size);
  int64_t want = 0;  // blocks of the forks so far
  __syncthreads();   // every thread has the counters
  for (int f0 = 0; f0 < a.F; f0 += kForkThreads * N) {
    Fork x[N];
    bool good[N], part[N];
    int32_t old[N];  // the last page's block, -1: none, or no block of the cache
    int own = 0;
#pragma unroll
    for (int j = 0; j < N; j++) {
      const int f = f0 + tid * N + j;
      good[j] = f < a.F && fork_of(a, f, x[j]);
      part[j] = good[j] && (x[j].len & ((1 << a.page_shift) - 1)) != 0;
      old[j] = part[j] ? a.table[int64_t(x[j].src) * a.width + x[j].whole] : -1;
    }
#pragma unroll
    for (int j = 0; j < N; j++) {
      if (old[j] < 0 || old[j] >= a.blocks) old[j] = -1;
      own += old[j] >= 0;  // takes a block
    }
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += t;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    int64_t rank = want + upto - own;
#pragma unroll
    for (int w = 0; w < kForkThreads / 32; w++) {
      if (w < warp) rank += s_sum[w];
      want += s_sum[w];
    }
    int32_t fresh[N];
#pragma unroll
    for (int j = 0; j < N; j++) {
      const int64_t at = first + rank;  // rank < avail <= ring_size
      fresh[j] = old[j] >= 0 && rank < avail ? a.ring[at < a.ring_size ? at : at - a.ring_size] : -1;
      if (old[j] >= 0 && rank >= avail) old[j] = -2;  // none left
      rank += old[j] != -1;
    }
#pragma unroll
    for (int j = 0; j < N; j++) {
      const int f = f0 + tid * N + j;
      if (f >= a.F) continue;
      const bool none = fresh[j] < 0 || fresh[j] >= a.blocks;
      if (!good[j] || (part[j] && none && old[j] != -2)) atomicOr(&g_status_kv_pages, DEV_BAD_INDEX);
      if (part[j]) a.table[int64_t(x[j].dst) * a.width + x[j].whole] = none ? -1 : fresh[j];
      a.from_blocks[f] = none ? -1 : old[j];
      a.to_blocks[f] = none ? -1 : fresh[j];
      a.lens_out[f] = !good[j] ? 0 : part[j] && none ? x[j].whole << a.page_shift : x[j].len;
    }
    __syncthreads();  // s_sum has been read
  }
  if (tid == 0) {
    const int64_t took = want < avail ? want : avail;
    a.ring_out[0] = head + took;
    a.ring_out[1] = tail;
    a.ring_out[2] = want - took;
  }
}

// The first CTA has the last pages; of the others each has one fork and kSegment entries of its row.  Forks of 62 whole pages
// and a partial one take 2.9 us for 4 (three dependent reads: lengths, table, ring), 3.4 for 256, 12 for 4096 and 70 for
// 16384 (a million counts of shared pages); each fork's CTA counting those before it 2.9, 3.4, 40 and 533.
__global__ void __launch_bounds__(kForkThreads) kv_fork_kernel(KvForkArgs a) {
  if (blockIdx.x == 0) {
    if (blockIdx.y > 0) return;
    if (a.F <= kForkThreads) fork_parts<1>(a);
    else fork_parts<4>(a);
    return;
  }
  Fork x;
  if (!fork_of(a, int(blockIdx.x) - 1, x)) return;
  const int32_t* from = a.table + int64_t(x.src) * a.width;
  int32_t* to = a.table + int64_t(x.dst) * a.width;
  const int j0 = blockIdx.y * kSegment, end = min(x.whole, j0 + kSegment);
  for (int j = j0 + threadIdx.x; j < end; j += kForkThreads) {
    int32_t b = -1;
    if (j < x.gap || j >= x.gap_end) {  // what was given up may be the ring's or another request's by now
      b = from[j];
      if (b < 0 || b >= a.blocks) {
        atomicOr(&g_status_kv_pages, DEV_BAD_INDEX);
        b = -1;
      } else {
        atomicAdd(a.refs + b, 1);
      }
    }
    to[j] = b;
  }
}

// One owner fewer for the blocks of entries j, j + step, .. of a range of pages.
__device__ __forceinline__ void unref(const KvFreeArgs& a, int f, int j, int end, int step, bool first_thread) {
  const int r = __ldg(a.rows + f), from = __ldg(a.first + f), to = __ldg(a.end + f);
  if (r < 0 || r >= a.R || from < 0 || to > a.width) {
    if (first_thread) atomicOr(&g_status_kv_pages, DEV_BAD_INDEX);
    return;
  }
  const int32_t* row = a.table + int64_t(r) * a.width;
  end = min(end, to);
  for (; j < end; j += step) {
    if (j < from) continue;
    const int32_t b = __ldg(row + j);
    if (b >= a.blocks) atomicOr(&g_status_kv_pages, DEV_BAD_INDEX);
    else if (b >= 0) atomicSub(a.refs + b, 1);
  }
}

// One range and kSegment entries of its row a CTA.
__global__ void __launch_bounds__(kThreads) kv_unref_kernel(KvFreeArgs a) {
  const int j0 = blockIdx.y * kSegment;
  unref(a, blockIdx.x, j0 + threadIdx.x, j0 + kSegment, kThreads, blockIdx.y == 0 && threadIdx.x == 0);
}

// Blocks whose count is negative, in ascending order, to the ring: one cluster, a run of steps of 32 blocks a
// warp.  `inside`: before that, the ranges are given up here, a warp a range.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kScan) kv_collect_kernel(KvFreeArgs a, bool inside) {
  namespace cg = cooperative_groups;
  __shared__ int s_warp[kScan / 32];
  __shared__ int s_total;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = int(cluster.block_rank());
  const int64_t warps = kCluster * (kScan / 32), mine = int64_t(warp) * kCluster + rank;
  const int64_t head = a.ring_in[0], tail = a.ring_in[1], lacked = a.ring_in[2];
  if (inside) {
    for (int f = int(mine); f < a.F; f += int(warps)) unref(a, f, lane, a.width, 32, lane == 0);
    cluster.sync();
  }
  const int64_t steps = (a.blocks + 31) / 32, per = (steps + warps - 1) / warps;
  const int64_t w0 = int64_t(rank) * (kScan / 32) + warp;  // runs in the order of CTAs, then warps
  const int64_t s0 = min(steps, w0 * per), s1 = min(steps, s0 + per);
  int count = 0;
  for (int64_t s = s0; s < s1; s += 4) {
    int c[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int64_t b = (s + i) * 32 + lane;
      c[i] = s + i < s1 && b < a.blocks ? __ldcg(a.refs + b) : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (c[i] < -1) atomicOr(&g_status_kv_pages, DEV_BAD_INDEX);  // given up more often than owned
      count += __popc(__ballot_sync(0xFFFFFFFFu, c[i] < 0));
    }
  }
  if (lane == 0) s_warp[warp] = count;
  __syncthreads();
  if (tid == 0) {
    int t = 0;
    for (int w = 0; w < kScan / 32; w++) t += s_warp[w];
    s_total = t;
  }
  cluster.sync();
  int64_t before = 0, total = 0;
  for (int c = 0; c < kCluster; c++) {
    const int t = *cluster.map_shared_rank(&s_total, c);
    if (c < rank) before += t;
    total += t;
  }
  for (int w = 0; w < warp; w++) before += s_warp[w];
  if (count > 0) {
    int64_t place = in_ring(tail + before, a.ring_size);
    for (int64_t s = s0; s < s1; s++) {
      const int64_t b = s * 32 + lane;
      const bool gone = b < a.blocks && __ldcg(a.refs + b) < 0;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, gone);
      if (gone) {
        const int64_t at = place + __popc(m & ((1u << lane) - 1u));
        a.ring[at < a.ring_size ? at : in_ring(at, a.ring_size)] = int32_t(b);
        a.refs[b] = 0;
      }
      place += __popc(m);
      if (place >= a.ring_size) place = in_ring(place, a.ring_size);
    }
  }
  cluster.sync();  // every CTA has read the counters and the totals
  if (rank == 0 && tid == 0) {
    a.ring_out[0] = head;
    a.ring_out[1] = tail + total;
    a.ring_out[2] = lacked;
  }
}

// Whole blocks: the codes and scales of all heads of one lie in one piece each.  A CTA has the same few words of
// every pair's blocks, and writes when it has read them all, so blocks may be read and written in one call (a
// list of moves).  2^log2_words words of 16 bytes: eight, a line of memory; more for few pairs, to fill the CTA, and
// fewer for many, so that several CTAs fit an SM (1000 pairs of 128 rows, 8 heads: eight words 78 us, four 55, 5.0 TB/s).
// 512 threads: 200 pairs of 16 rows 3.8 us, of 64 rows 6.3; in their time 256 threads 4.6 and 6.4, 512 3.9 and 6.7, 1024 3.6 and 8.2.
// Of several pairs that write one block the last is kept: each looks itself up by its block in `last`, an open table
// of at least two places a pair, which lies where the words are put afterwards.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(KvPages c, const int32_t* from, const int32_t* to, int n, int log2_words, int code_words,
                                                           int sf_words, int log2_last) {
  extern __shared__ uint4 stage[];
  const int count = n << log2_words, mask = (1 << log2_words) - 1;
  int* last = reinterpret_cast<int*>(stage);
  const int places = 1 << log2_last;
  int2* pairs = reinterpret_cast<int2*>(stage + count);  // the table, less than 16 bytes a pair, ends before
  for (int i = threadIdx.x; i < n; i += kCopyThreads) {
    int2 p = make_int2(__ldg(from + i), __ldg(to + i));
    if (p.x >= c.blocks || p.y >= c.blocks) {
      if (blockIdx.x == 0 && p.x >= 0 && p.y >= 0) atomicOr(&g_status_kv_pages, DEV_BAD_INDEX);
      p.x = -1;
    }
    if (p.y < 0) p.x = -1;
    pairs[i] = p;
  }
  for (int i = threadIdx.x; i < places; i += kCopyThreads) last[i] = -1;
  __syncthreads();
  // the place of a block: the first one from its hash on that `at` says is its
  auto find = [&](int32_t block, auto&& at) {
    uint32_t h = (uint32_t(block) * 0x9E3779B1u) >> (32 - log2_last);
    for (int t = 0; t < places && !at(last + h); t++) h = (h + 1) & uint32_t(places - 1);
  };
  for (int i = threadIdx.x; i < n; i += kCopyThreads) {
    const int2 pair = pairs[i];
    if (pair.x < 0) continue;
    find(pair.y, [&](int* p) {
      const int j = atomicCAS(p, -1, i);
      if (j >= 0 && pairs[j].y != pair.y) return false;
      if (j >= 0) atomicMax(p, i);
      return true;
    });
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kCopyThreads) {
    const int2 pair = pairs[i];
    if (pair.x < 0) continue;
    find(pair.y, [&](int* p) {
      if (pairs[*p].y != pair.y) return false;
      if (*p != i) pairs[i].x = -1;
      return true;
    });
  }
  __syncthreads();
  // word i of the CTA in a block: which of the four arrays, and where
  auto place = [&](int i, int32_t block) -> uint4* {
    int w = (int(blockIdx.x) << log2_words) + (i & mask);
    const bool codes = w < 2 * code_words;
    if (!codes) w -= 2 * code_words;
    const int words = codes ? code_words : sf_words;
    const bool second = w >= words;
    if (second) w -= words;
    if (w >= words) return nullptr;
    uint4* p = reinterpret_cast<uint4*>(codes ? (second ? c.v : c.k) : (second ? c.v_sf : c.k_sf));
    return p + int64_t(block) * words + w;
  };
#pragma unroll 4
  for (int i = threadIdx.x; i < count; i += kCopyThreads) {
    const int2 pair = pairs[i >> log2_words];
    const uint4* src = pair.x < 0 ? nullptr : place(i, pair.x);
    if (src) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(stage + i)), "l"(src) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < count; i += kCopyThreads) {
    const int2 pair = pairs[i >> log2_words];
    uint4* dst = pair.x < 0 ? nullptr : place(i, pair.y);
    if (dst) *dst = stage[i];
  }
}

}  // namespace

cudaError_t launch_kv_fork(const KvForkArgs& a, cudaStream_t st) {
  clear_stale_error();
  const dim3 grid(unsigned(a.F + 1), unsigned((a.width + kSegment - 1) / kSegment));
  kv_fork_kernel<<<grid, kForkThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv_free(const KvFreeArgs& a, cudaStream_t st) {
  clear_stale_error();
  // few entries: in the one cluster that collects, which saves a launch
  const bool inside = int64_t(a.F) * a.width <= kInside;
  if (!inside) {
    kv_unref_kernel<<<dim3(unsigned(a.F), unsigned((a.width + kSegment - 1) / kSegment)), kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  kv_collect_kernel<<<kCluster, kScan, 0, st>>>(a, inside);
  return cudaGetLastError();
}

cudaError_t launch_kv_copy(const KvPages& c, const int32_t* from, const int32_t* to, int n, cudaStream_t st) {
  clear_stale_error();
  static std::atomic<unsigned long long> done{0};
  constexpr int kBytes = kKvCopyMost * (16 + 8);  // words, and pairs of the largest call
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kv_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  });
  if (e != cudaSuccess) return e;
  int log2_words = 3;
  while (log2_words > 1 && (int64_t(n) << log2_words) > 4096) log2_words--;
  while (log2_words > 0 && (int64_t(n) << log2_words) > kKvCopyMost) log2_words--;
  while (log2_words < 6 && (int64_t(n) << log2_words) < kCopyThreads) log2_words++;
  int log2_last = 1;
  while ((1 << log2_last) < 2 * n) log2_last++;
  const size_t shared = (size_t(n) << log2_words) * 16 + size_t(n) * 8;
  const int codes = c.H * c.page * 4, sf = c.H * c.page / (c.fmt == 0 ? 4 : 2);
  const int64_t words = 2 * (int64_t(codes) + sf);
  const unsigned grid = unsigned((words + (1 << log2_words) - 1) >> log2_words);
  kv_copy_kernel<<<grid, kCopyThreads, shared, st>>>(c, from, to, n, log2_words, codes, sf, log2_last);
  return cudaGetLastError();
}

unsigned read_status_kv_pages(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv_pages, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_kv_pages, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
