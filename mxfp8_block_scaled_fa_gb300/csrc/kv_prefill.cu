// kv_prefill.cu -- attention over the 4-bit key/value cache for many query rows of a
// request: prompts and chunks of prompts.  The arithmetic of kv_attn.cu (q, K, V and
// P in binary16, exact products, fp32 sums and softmax) on the 5th-generation tensor
// core.
//
// Work.  An item is (request, key head, block of 256 query rows), a row being a query
// head of the group at a token; its keys come in tiles of 128, up to the last one a
// row sees.  As in kv_attn.cu the tiles of all items form one line that is cut
// into equal runs, one per CTA (one CTA per SM); an item cut by a border leaves
// partial (m, l, O) records that kv_prefill_join_kernel joins.  A kernel of one CTA
// writes the requests' places on the line first.
//
// CTA: 16 warps.
//   warps 0, 2   tcgen05 issuers of the row tiles A and B; warp 0 owns the TMEM
//   warp 1       walks the run and publishes its items (two-entry ring)
//   warps 4-7    softmax of rows 0..127 (tile A): thread = row = TMEM lane; and tile A's
//                queries of the next item, as soon as its last S is done
//   warps 8-11   the same of rows 128..255 (tile B)
//   warps 12-15  conversion: 4-bit rows of K and V from global memory (held in
//                registers half a tile ahead) to binary16 tiles in shared memory, 128B
//                swizzle, two of each
// K is read as the K-major and V as the MN-major operand of the same layout: [channel
// half][key][64 channels].
//   TMEM (512 columns): S_A, S_B, O_A, O_B of 128.  S_X is two halves of 64 keys; a
//   half's P (32 columns of binary16 pairs) replaces its S, and the half's next S is
//   issued behind the product that reads P.  So the tensor core works on one half
//   while the softmax warps are at the other, of both tiles.
//
// What bounds it.  A tile of 128 keys x 256 rows is 4 x 512 cycles of the tensor core, and
// half as long for the 32768 exponentials.  The products of 64 keys read Q again for
// each half (6 KB of shared memory in 32 cycles, where 128 B a cycle is the most), and
// take 50 to 90 cycles each instead of 32.  Chunks of 2048 and 1687 tokens over 8192 and
// 5331 keys, 8 key heads, G = 4, NVFP4: 304 us, 1200 TFLOP/s, of which the main
// kernel 285 us; about 3300 cycles a tile (issuers: P V 750, S 1400, waits), and
// 12000 cycles between items, when the softmax warps bring the next queries (half of
// them) and write O.  Other forms of it, same case: whole S products of 128 keys and
// one issuer, softmax, P V and S in turn, 347 us; these with two issuers 360 to 407 us;
// halves with one issuer 457 us (a product is issued in 40 to 55 cycles, a commit in
// 100); conversion with coalesced loads (four lanes a row) 435 against 379 us, as the
// swizzled stores then cost more; O written through shared memory by rows, 315 against
// 312 us.  For items of up to 128 rows both softmax groups on the same rows, each with
// half of the keys, 137 against 117 us for 24 x 64 rows over 6000 keys.  Launched ahead
// of the kernels they wait for, the five kernels of a call take 313 instead of 319 us
// from a stream (310 from a graph, either way).  These are figures of their time, against 309 us in the end; the
// issuers' loops over items, no longer than the call's tokens need, then made it 304.
//
// Windows and prefixes (KvKind, as in kv_attn.cu).  With a window an item's keys are the tiles of the sinks and those from its
// first row's window on; the tiles between are no part of the line, and what a row does not see of the others is masked by
// bits.  The chunks above with a window of 1024 and 64 sinks: 106 us, 8.5 tiles' worth of keys in 10.5 tiles an item, and
// the 12000 cycles between items on 472 items; a half whose keys no row of a warp sees is computed like the others
// (left out: no change).  A prefix takes about 21 us for up to eight tiles, of which 4 pass until the item is known, 3 for the
// queries, 0.85 a tile, and 5 for the records, as each thread stores its row (rows side by side: 2, and 2 us more in the join).
#include "kv_fp4.cuh"
#include "mx_ptx.cuh"
#include "mxfa_internal.h"

#include <cmath>

namespace mxfa {

static __device__ unsigned g_status_kv_prefill;

namespace kvp {

constexpr int TILE = kPrefillTile;       // keys of a tile, rows of an MMA
constexpr int ROWS = kPrefillRows;       // query rows of an item
constexpr int OP_BYTES = TILE * 256;     // 128 rows x 128 binary16
// What an item costs beside its tiles, in tiles: 1, 2, 3 and 4 took 319, 317, 314 and 312
// us for the prompts above.
constexpr int kItemTiles = kPrefillItemTiles;
// Least units of a run: a shorter one costs more to join than it saves.  Of prefixes 4, 6, 8 and 10 units took 52, 51, 47 and
// 45 us for one of 8192 keys and 64 requests with up to 1024 keys behind it (whose kernel gets the other SMs), 29, 27, 30
// and 32 us for six of up to 3000 keys and 30 requests with up to 300, and 6, 8 and 10 units 32, 35 and 40 us for one of
// 8192 keys and next to nothing behind it.
constexpr int kMinUnits = 6;
constexpr float kOffset = 8.0f, kLazy = 6.0f;  // as in kv_attn.cu

constexpr int OFF_Q = 0;                           // tiles A, B
constexpr int OFF_K = OFF_Q + 2 * OP_BYTES;        // two stages
constexpr int OFF_V = OFF_K + 2 * OP_BYTES;        // two stages
constexpr int OFF_CS = OFF_V + 2 * OP_BYTES;       // float [256]: row scales
constexpr int OFF_NAN = OFF_CS + ROWS * 4;     // u8 [4][128]: NaN blocks of V of a tile's keys
constexpr int OFF_BAD = OFF_NAN + 4 * TILE;        // u32 [4][4]: keys that are not there
constexpr int OFF_FLAG = OFF_BAD + 64;             // u32 [4][4]: per conversion warp, 1: NaN blocks, 2: missing keys
constexpr int OFF_ITEM = OFF_FLAG + 64;            // Item [2]
constexpr int OFF_BAR = OFF_ITEM + 128;
enum {
  B_QFULL = 0, B_KFULL = B_QFULL + 2, B_KEMPTY = B_KFULL + 2, B_VFULL = B_KEMPTY + 2, B_VEMPTY = B_VFULL + 2,
  B_SFULL = B_VEMPTY + 2, B_PFULL = B_SFULL + 4, B_ODONE = B_PFULL + 4, B_IFULL = B_ODONE + 4, B_IEMPTY = B_IFULL + 2,
  B_TEAR = B_IEMPTY + 2, NBAR
};
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
constexpr int READERS = 2 + 8 + 4;                 // warps that read an item

constexpr uint32_t COL_S = 0, COL_O = 256;         // + 128 * tile
constexpr int NTHREADS = 512;
constexpr int REG_ISSUE = 56, REG_SOFTMAX = 184, REG_CONVERT = 88;
static_assert(128 * (REG_ISSUE + 2 * REG_SOFTMAX + REG_CONVERT) <= NTHREADS * 128, "register split exceeds the launch allocation");

struct Item {
  int r, h, row0, rows;
  int q0, n, kv, t0;
  int na, nb;       // tiles of A and of B in this part
  int slot;         // -1: the whole item, else partial record
  int lo, hi, at, jump;  // as in Request
  int parts;        // of the item that begins here: CTAs that hold one (0: this one alone)
};
static_assert(sizeof(Item) == 64, "an item record");

struct Header {
  int r, h, row0;   // the item that begins in this CTA's run and ends behind it
  int parts;        // number of further CTAs that hold a part of it; 0: none
};
struct Partial {
  float o[ROWS][128];
  float m[ROWS], l[ROWS];
};

__host__ __device__ inline size_t line_bytes(int R) { return (size_t(R + 1) * 8 + 255) & ~size_t(255); }
__host__ __device__ inline size_t header_bytes(int ctas) { return (size_t(ctas) * sizeof(Header) + 255) & ~size_t(255); }

// kind::f16, binary16 operands, fp32 accumulation; issued by an elected lane of a
// converged warp.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss_w(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts_w(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// A request whose rows belong here: more than a.split_rows of them, offsets and
// lengths within their tables (a failed check leaves n = 0).
// kWindow, kTail: keys lo .. hi - 1 are in no row's sight (of an item, as item_of() sets them); the tiles that hold
// nothing else, `jump` keys of them from key `at` on, are left out of the item's tiles.  kTail, where prefixes are not
// shared after all: hi = 0, and keys before lo are those of the group's first request.
struct Request {
  int q0, n, kv;
  int lo, hi, at, jump;
};
__device__ __forceinline__ void hide(Request& x, int lo, int hi) {
  x.lo = lo, x.hi = hi;
  x.at = (lo + TILE - 1) / TILE * TILE;
  x.jump = max(0, hi / TILE * TILE - x.at);
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
    x.n = int64_t(n) * a.G > a.split_rows ? n : 0;
    return x;
  }
  const int64_t b = __ldg(a.cu_q + r), e = __ldg(a.cu_q + r + 1);
  const int kv = __ldg(a.kv_lens + r);
  const int64_t most = int64_t(a.width) << a.c.page_shift;
  if (b < 0 || e < b || e > a.total_q || e - b > a.max_q || kv < 0 || kv > most) {
    atomicOr(&g_status_kv_prefill, DEV_BAD_INDEX);
    x.q0 = x.n = x.kv = 0;
    return x;
  }
  x.q0 = int(b);
  x.n = (e - b) * a.G > a.split_rows ? int(e - b) : 0;
  x.kv = kv;
  if constexpr (KIND == kTail) {
    const int p = __ldg(a.prefix + r);  // negative: of a group that is none
    if (p > 0 && e > b && kv - (e - b) < p) atomicOr(&g_status_kv_prefill, DEV_BAD_INDEX);
    if (p < 0 || kv - (e - b) < p) x.n = 0;
    if (x.n > 0) {
      if (__ldg(a.share)) hide(x, 0, p);
      else x.lo = p;
    }
  }
  return x;
}
// What the item of rows row0 on leaves out.
template <int KIND>
__device__ __forceinline__ void item_of(const KvAttnArgs& a, Request& x, int row0) {
  if constexpr (KIND == kWindow) {
    const int lo = int(max(int64_t(0), int64_t(x.kv) - x.n + row0 / a.G - a.window + 1));
    hide(x, min(a.sinks, lo), lo);
  }
}
// Keys that the last of the rows before `row_end` sees.
__device__ __forceinline__ int keys_of(const KvAttnArgs& a, const Request& x, int row_end) {
  return a.causal ? max(0, x.kv - x.n + (row_end - 1) / a.G + 1) : x.kv;
}
__device__ __forceinline__ int tiles_of(const KvAttnArgs& a, const Request& x, int row0) {
  return max(1, (keys_of(a, x, min(row0 + ROWS, x.n * a.G)) - x.jump + TILE - 1) / TILE);
}

// line[r] = units (tiles, and kItemTiles per item) of the requests before r.
template <int KIND>
__global__ void __launch_bounds__(512) kv_prefill_line_kernel(KvAttnArgs a, int64_t* line) {
  __shared__ int64_t s_sum[16];
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t base = 0;
  for (int r0 = 0; r0 < a.R; r0 += 512) {
    const int r = r0 + threadIdx.x;
    int64_t u = 0;
    Request x;
    x.q0 = x.n = x.kv = x.lo = x.hi = x.at = x.jump = 0;
    if (r < a.R) x = request_of<KIND>(a, r);
    // a block of rows a lane, of the warp's requests one after another
    for (unsigned left = __ballot_sync(0xFFFFFFFFu, x.n > 0); left; left &= left - 1) {
      const int who = __ffs(left) - 1;
      Request y;
      y.q0 = 0;
      y.n = __shfl_sync(0xFFFFFFFFu, x.n, who), y.kv = __shfl_sync(0xFFFFFFFFu, x.kv, who);
      y.lo = y.hi = y.at = 0, y.jump = __shfl_sync(0xFFFFFFFFu, x.jump, who);
      int64_t all = 0;
      for (int row0 = lane * ROWS; row0 < y.n * a.G; row0 += 32 * ROWS) {
        item_of<KIND>(a, y, row0);
        all += tiles_of(a, y, row0) + kItemTiles;
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
      if (lane == who) u = all * a.c.H;
    }
    int64_t v = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    int64_t before = base, all = 0;
    for (int w = 0; w < 16; w++) {
      if (w < warp) before += s_sum[w];
      all += s_sum[w];
    }
    if (r < a.R) line[r] = before + v - u;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) line[a.R] = base;
  // it runs beside kv_attn_kernel, and its end stands for that one's too
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Bits 0 .. n - 1 of 64.
__device__ __forceinline__ uint64_t below(int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; }

template <int KIND, int FMT>
__global__ void __launch_bounds__(NTHREADS, 1) kv_prefill_kernel(const __grid_constant__ KvAttnArgs a, const int64_t* line,
                                                                 Header* headers, Partial* partials) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_addr);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = base + OFF_BAR;
  auto BAR = [&](int i) { return bar0 + 8u * uint32_t(i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + OFF_MISC + 8);
  unsigned* status = &g_status_kv_prefill;

  if (KIND != kPrefix) asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < 2; s++) {
      mbar_init(BAR(B_QFULL + s), 4);
      mbar_init(BAR(B_KFULL + s), 4);
      mbar_init(BAR(B_KEMPTY + s), 2);
      mbar_init(BAR(B_VFULL + s), 4);
      mbar_init(BAR(B_VEMPTY + s), 2);
      mbar_init(BAR(B_IFULL + s), 1);
      mbar_init(BAR(B_IEMPTY + s), READERS);
    }
    for (int s = 0; s < 4; s++) {  // tile, half of the keys
      mbar_init(BAR(B_SFULL + s), 1);
      mbar_init(BAR(B_PFULL + s), 4);
      mbar_init(BAR(B_ODONE + s), 1);
    }
    mbar_init(BAR(B_TEAR), 2);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the line, and what runs before it
  // the kernel behind the prefixes' reads what was written before this one
  if (KIND == kPrefix) asm volatile("griddepcontrol.launch_dependents;");
  // by the scheduler's lane, which may replace it: no barrier follows that would order two threads
  if (!kRecords<KIND> && warp == 1 && lane == 0) headers[blockIdx.x].parts = 0;
  const int64_t total = __ldcg(line + a.R);
  if (total == 0) {  // no request with that many rows
    if (warp == 0) tmem_dealloc(tmem, 512);
    return;
  }
  constexpr bool kHides = KIND == kWindow || KIND == kTail;
  // CTAs with a run: as many as it is worth, and for prefixes one an item at least
  auto runs = [&]() -> int64_t {
    int64_t most = (total + kMinUnits - 1) / kMinUnits;
    if (KIND == kPrefix) most = max(most, int64_t(__ldcg(a.prefix + a.R)));
    return min(most, int64_t(gridDim.x));
  };
  if (kRecords<KIND> && int64_t(blockIdx.x) >= runs()) {  // makes room
    if (warp == 0) tmem_dealloc(tmem, 512);
    return;
  }
  const Item* items = reinterpret_cast<const Item*>(smem + OFF_ITEM);
  // whole warp: waits for item i of the run and reads it; a part with rows == 0 ends the run
  auto take = [&](int i, Item& it, bool& ok) {
    ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(BAR(B_IFULL + (i & 1)), (i >> 1) & 1, abort_flag, status));
    it.rows = 0;
    if (ok) {
      const volatile Item* v = items + (i & 1);
      it.r = v->r, it.h = v->h, it.row0 = v->row0, it.rows = v->rows;
      it.q0 = v->q0, it.n = v->n, it.kv = v->kv, it.t0 = v->t0;
      it.na = v->na, it.nb = v->nb, it.slot = v->slot;
      if (kHides) it.lo = v->lo, it.hi = v->hi, it.at = v->at, it.jump = v->jump;
      if (kRecords<KIND>) it.parts = v->parts;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(B_IEMPTY + (i & 1)));
    return ok && it.rows > 0;
  };
  // whole warp: waits for a phase.  The test alone costs a third of a try_wait on a
  // completed barrier, the common case (prompts 330 -> 318 us with it in the issuers).
  auto wait_all = [&](uint32_t bar, uint32_t par) {
    if (__all_sync(0xFFFFFFFFu, mbar_test(bar, par))) return true;
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, par, abort_flag, status)) != 0;
  };
  auto warp_arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_ISSUE));
    if (warp == 0 || warp == 2) {
      // --------------------------------------------------------------- issuers
      warp_converged();
      const int x = warp >> 1;  // tile A or B
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      // S_X = Q_X K^T for half h of running tile kt's keys
      auto issue_s = [&](int h, int kt) {
        const uint64_t dq = smem_desc(base + OFF_Q + x * OP_BYTES, 16, 1024, 2);
        const uint64_t dk = smem_desc(base + OFF_K + (kt & 1) * OP_BYTES, 16, 1024, 2) + uint64_t(h * (OP_BYTES / 64));
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const uint64_t off = uint64_t((k >> 2) * (OP_BYTES / 32) + (k & 3) * 2);  // channel half, 32 bytes of it
          mma_ss_w(tm + COL_S + 128 * x + 64 * h, dq + off, dk + off, idesc_f16(128, 64, 0), k > 0);
        }
        tc_commit_w(BAR(B_SFULL + 2 * x + h));
      };
      // O_X (+)= P_X V for half h
      auto issue_pv = [&](int h, int kt, bool first) {
        const uint64_t dv = smem_desc(base + OFF_V + (kt & 1) * OP_BYTES, OP_BYTES / 2, 1024, 2) + uint64_t(h * 512);
#pragma unroll
        for (int k = 0; k < 4; k++)  // 16 keys: 2048 bytes of each channel half
          mma_ts_w(tm + COL_O + 128 * x, tm + COL_S + 128 * x + 64 * h + 8 * k, dv + uint64_t(128 * k), idesc_f16(128, 128, 1),
                   !first || k > 0);
        tc_commit_w(BAR(B_ODONE + 2 * x + h));
      };
      int kt = 0;             // tiles passed
      int sn = 0, qn = 0;     // S products and items of this tile so far
      bool ok = true;
      // The loops over items have trip counts of the call's arguments (a.item_loops^3 is no fewer than
      // a run can have, by the tokens of the call) and skip their turns once the run is over: a loop that ended on
      // a loaded item would not be warp-uniform to the compiler, and the issue code in it took 130
      // cycles a product instead of 64.  A skipped turn takes 60 ns: four loops of 64, whatever the
      // call, cost it 16 us.
      bool over = false;
      int i = 0;
#pragma unroll 1
      for (int l0 = 0; l0 < a.item_loops; l0++) {
        if (over) continue;
#pragma unroll 1
      for (int l1 = 0; l1 < a.item_loops; l1++) {
        if (over) continue;
#pragma unroll 1
      for (int l2 = 0; l2 < a.item_loops; l2++) {
        if (over) continue;
        Item it;
        if (!take(i++, it, ok)) {
          over = true;
          continue;
        }
        const int n = x ? it.nb : it.na, nmax = max(it.na, it.nb);
        if (n > 0) {
          ok = wait_all(BAR(B_QFULL + x), uint32_t(qn) & 1) && wait_all(BAR(B_KFULL + (kt & 1)), (kt >> 1) & 1);
          tc_fence_after();
          if (ok) {
            issue_s(0, kt);
            issue_s(1, kt);
            tc_commit_w(BAR(B_KEMPTY + (kt & 1)));
          }
          qn++;
        }
        // P V and the next S of a half one after the other: the tensor core runs them in this
        // order, so S overwrites P only when it has been read
#pragma unroll 1
        for (int j = 0; ok && j < n; j++) {
          const int kj = kt + j;
          const bool next = j + 1 < n;
          // K(j + 1) is converted after V(j) by the same warps, so its barrier covers both
          ok = next ? wait_all(BAR(B_KFULL + ((kj + 1) & 1)), ((kj + 1) >> 1) & 1) : wait_all(BAR(B_VFULL + (kj & 1)), (kj >> 1) & 1);
#pragma unroll 1
          for (int h = 0; ok && h < 2; h++) {
            ok = wait_all(BAR(B_PFULL + 2 * x + h), uint32_t(sn + j) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_pv(h, kj, j + h == 0);
            if (next) issue_s(h, kj + 1);
          }
          if (ok) {
            tc_commit_w(BAR(B_VEMPTY + (kj & 1)));
            if (next) tc_commit_w(BAR(B_KEMPTY + ((kj + 1) & 1)));
          }
        }
        // tiles that only the other rows need: released once they are there
#pragma unroll 1
        for (int j = n; ok && j < nmax; j++) {
          const int kj = kt + j;
          ok = wait_all(BAR(B_KFULL + (kj & 1)), (kj >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(BAR(B_KEMPTY + (kj & 1)));
          ok = ok && wait_all(BAR(B_VFULL + (kj & 1)), (kj >> 1) & 1);
          if (ok && lane == 0) mbar_arrive(BAR(B_VEMPTY + (kj & 1)));
          __syncwarp();
        }
        kt += nmax;
        sn += n;
        if (!ok) over = true;
      }
      }
      }
      // every product has retired before TMEM is released
      tc_commit_w(BAR(B_TEAR));
      const unsigned long long t0 = global_ns();
      while (!mbar_try_wait_sleep(BAR(B_TEAR), 0))
        if (global_ns() - t0 > kWaitLimitNs) break;
      __syncwarp();
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------------- scheduler
      const int64_t C = runs();
      const int64_t run = total / C, extra = total - run * C;  // the first `extra` CTAs take one unit more
      int64_t pos = run * blockIdx.x + min(extra, int64_t(blockIdx.x));
      int64_t end = pos + run + (int64_t(blockIdx.x) < extra ? 1 : 0);
      if (int64_t(blockIdx.x) >= C) pos = end = 0;
      int lo = 0, hi = a.R;  // the request with line[lo] <= pos < line[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(line + mid) <= pos) lo = mid;
        else hi = mid;
      }
      int r = lo, i = 0;
      auto publish = [&](const Item& it) -> bool {
        // beyond the issuers' turns: of offsets that are none, whose requests hold more rows than the call has tokens
        if (i >= a.item_most && it.rows > 0) {
          atomicOr(status, DEV_BAD_INDEX);
          return false;
        }
        if (i >= 2 && !mbar_wait(BAR(B_IEMPTY + (i & 1)), ((i >> 1) - 1) & 1, abort_flag, status)) return false;
        volatile Item* v = reinterpret_cast<volatile Item*>(smem + OFF_ITEM) + (i & 1);
        v->r = it.r, v->h = it.h, v->row0 = it.row0, v->rows = it.rows;
        v->q0 = it.q0, v->n = it.n, v->kv = it.kv, v->t0 = it.t0;
        v->na = it.na, v->nb = it.nb, v->slot = it.slot;
        if (kHides) v->lo = it.lo, v->hi = it.hi, v->at = it.at, v->jump = it.jump;
        if (kRecords<KIND>) v->parts = it.parts;
        mbar_arrive(BAR(B_IFULL + (i & 1)));
        i++;
        return true;
      };
      bool ok = true;
      while (ok && pos < end && r < a.R) {
        const int64_t lr = __ldcg(line + r), next_r = __ldcg(line + r + 1);
        if (pos >= next_r) {
          r++;
          continue;
        }
        Request x = request_of<KIND>(a, r);
        const int64_t per_head = (next_r - lr) / a.c.H;
        int h = int((pos - lr) / per_head);
        int64_t at = lr + h * per_head;  // start of the item that is looked at
        int row0 = 0;
        // items of the request from pos on: head by head, block by block
        while (ok && pos < end && h < a.c.H) {
          if (row0 >= x.n * a.G) {
            row0 = 0;
            h++;
            continue;
          }
          item_of<KIND>(a, x, row0);
          const int tiles = tiles_of(a, x, row0), units = tiles + kItemTiles;
          if (pos >= at + units) {
            at += units;
            row0 += ROWS;
            continue;
          }
          const int u0 = int(pos - at), u1 = int(min(int64_t(units), u0 + (end - pos)));
          const int t0 = max(0, u0 - kItemTiles), t1 = max(0, u1 - kItemTiles);
          pos += u1 - u0;
          if (t1 > t0) {
            Item it;
            it.r = r, it.h = h, it.row0 = row0;
            it.rows = min(ROWS, x.n * a.G - row0);
            it.q0 = x.q0, it.n = x.n, it.kv = x.kv, it.t0 = t0;
            it.lo = x.lo, it.hi = x.hi, it.at = x.at, it.jump = x.jump;
            const int va = (keys_of(a, x, row0 + min(TILE, it.rows)) - x.jump + TILE - 1) / TILE;
            const int vb = it.rows > TILE ? (keys_of(a, x, row0 + it.rows) - x.jump + TILE - 1) / TILE : 0;
            it.na = max(0, min(va, t1) - t0);
            it.nb = max(0, min(vb, t1) - t0);
            it.slot = t0 > 0 ? 2 * int(blockIdx.x) : t1 < tiles ? 2 * int(blockIdx.x) + 1 : -1;
            it.parts = 0;
            if (t0 == 0 && t1 < tiles) {
              const int64_t last = at + units - 1, larger = extra * (run + 1);
              Header hd;
              hd.r = r, hd.h = h, hd.row0 = row0;
              hd.parts = int(last < larger ? last / (run + 1) : extra + (last - larger) / run) - int(blockIdx.x);
              it.parts = hd.parts + 1;
              if (!kRecords<KIND>) headers[blockIdx.x] = hd;
            }
            ok = publish(it);
          }
        }
        r++;
      }
      {
        Item none;
        none.r = none.h = none.row0 = none.rows = none.q0 = none.n = none.kv = none.t0 = none.na = none.nb = none.slot = 0;
        none.lo = none.hi = none.at = none.jump = none.parts = 0;
        publish(none);
      }
    }
    __syncwarp();
  } else if (warp >= 12) {
    // ---------------------------------------------------------------- conversion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_CONVERT));
    const int t = tid - 384;  // row of the tile
    const int cw = warp - 12;
    const uint32_t swz = uint32_t(t & 7) << 4;
    int kt = 0;
    bool ok = true;
    Item it;
    for (int i = 0; take(i, it, ok); i++) {
      const int nmax = max(it.na, it.nb);
      if (nmax == 0) continue;
      const int32_t* table = a.table + int64_t(KIND == kPrefix ? __ldg(a.starts + it.r) : it.r) * a.width;
      Request x;
      x.q0 = it.q0, x.n = it.n, x.kv = it.kv;
      const int keys = keys_of(a, x, it.row0 + it.rows);  // that some row sees
      // this thread's row of tile j of the part: codes and scales, K and V
      // What a load brings is first looked at half a tile later, or it would be waited for:
      // the table entry two tiles ahead, V's scales with K's row.
      uint4 kc[4], vc[4];
      uint2 ks, vs, next_vs;
      int64_t row;      // cache row of the tile's key, -1: none, -2: not in the cache
      int next_block;   // table entry of the next tile's key
      auto key_of = [&](int j) {
        const int place = (it.t0 + j) * TILE;
        return (kHides && place >= it.at ? place + it.jump : place) + t;
      };
      const int32_t* first_table = KIND == kTail && it.hi < it.lo ? a.table + int64_t(__ldg(a.starts + it.r)) * a.width : table;
      auto in_sight = [&](int key) { return key < keys && (!kHides || key < it.lo || key >= it.hi); };
      auto entry = [&](int j) -> int {
        const int key = key_of(j);
        return j < nmax && in_sight(key) ? __ldg((KIND == kTail && key < it.lo ? first_table : table) + (key >> a.c.page_shift)) : -1;
      };
      auto find = [&](int b, int j) -> int64_t {
        const int key = key_of(j);
        if (j >= nmax || !in_sight(key)) return -1;
        if (b < 0 || b >= a.c.blocks) return -2;
        return (int64_t(b) * a.c.H + it.h) * a.c.page + (key & (a.c.page - 1));
      };
      auto load_k = [&](int64_t at) {
#pragma unroll
        for (int w = 0; w < 4; w++) kc[w] = make_uint4(0, 0, 0, 0);
        ks = next_vs = make_uint2(0, 0);
        if (at >= 0) {
          const uint4* src = reinterpret_cast<const uint4*>(a.c.k + at * 64);
#pragma unroll
          for (int w = 0; w < 4; w++) kc[w] = __ldg(src + w);
          if (FMT == 0) {
            ks.x = __ldg(reinterpret_cast<const uint32_t*>(a.c.k_sf + at * 4));
            next_vs.x = __ldg(reinterpret_cast<const uint32_t*>(a.c.v_sf + at * 4));
          } else {
            ks = __ldg(reinterpret_cast<const uint2*>(a.c.k_sf + at * 8));
            next_vs = __ldg(reinterpret_cast<const uint2*>(a.c.v_sf + at * 8));
          }
        }
      };
      auto load_v = [&](int64_t at) {
#pragma unroll
        for (int w = 0; w < 4; w++) vc[w] = make_uint4(0, 0, 0, 0);
        if (at >= 0) {
          const uint4* src = reinterpret_cast<const uint4*>(a.c.v + at * 64);
#pragma unroll
          for (int w = 0; w < 4; w++) vc[w] = __ldg(src + w);
        }
      };
      row = find(entry(0), 0);
      load_k(row);
      load_v(row);
      next_block = entry(1);
      // a row of a tile: sixteen words of eight channels, chunk (16 bytes) w of 16
      auto put = [&](uint32_t tile, const uint4* c, const uint32_t* s2) {
        const uint32_t dst = tile + uint32_t(t) * 128u;
#pragma unroll
        for (int w = 0; w < 16; w++) {
          const uint4 q = c[w >> 2];
          const uint32_t word = (w & 3) == 0 ? q.x : (w & 3) == 1 ? q.y : (w & 3) == 2 ? q.z : q.w;
          const uint32_t sc = FMT == 0 ? s2[w >> 2] : s2[w >> 1];
          uint32_t hv[4];
          e2m1x8_to_f16(word, hv);
          st_shared_v4(dst + (w >> 3) * (OP_BYTES / 2) + ((uint32_t(w & 7) << 4) ^ swz), hmul2(hv[0], sc), hmul2(hv[1], sc),
                       hmul2(hv[2], sc), hmul2(hv[3], sc));
        }
      };
      // block scales as binary16 pairs of one value
      auto scales = [&](const uint2& b, uint32_t* s2) {
        if (FMT == 0) {
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const uint32_t byte = (b.x >> (8 * e)) & 0xFFu;
            s2[e] = e8m0_pair(byte, byte);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const uint32_t two = e4m3_pair((e < 2 ? b.x : b.y) >> (16 * (e & 1)));
            s2[2 * e] = __byte_perm(two, two, 0x1010);
            s2[2 * e + 1] = __byte_perm(two, two, 0x3232);
          }
        }
      };
      for (int j = 0; ok && j < nmax; j++, kt++) {
        const int st = kt & 1, f4 = kt & 3;
        // stage st held tile kt - 2; and when it is free, the softmax of tile kt - 4 is
        // done, whose flags are replaced
        if (kt >= 2) ok = wait_all(BAR(B_KEMPTY + st), ((kt >> 1) - 1) & 1);
        if (!ok) break;
        // NaN blocks of V: taken out of the product here, put into the rows that see the
        // key by their softmax threads; keys whose block is not in the cache
        uint32_t nan = 0;
        vs = next_vs;
        if (FMT == 0) {
          const uint32_t m = __vcmpeq4(vs.x, 0xFFFFFFFFu);
          vs.x &= ~m;
          nan = ((m & 1u) * 3u) | (((m >> 8) & 1u) * 12u) | (((m >> 16) & 1u) * 48u) | ((m >> 24) & 1u) * 192u;
        } else {
          const uint32_t m0 = __vcmpeq4(vs.x & 0x7F7F7F7Fu, 0x7F7F7F7Fu), m1 = __vcmpeq4(vs.y & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
          vs.x &= ~m0;
          vs.y &= ~m1;
#pragma unroll
          for (int e = 0; e < 4; e++) nan |= (((m0 >> (8 * e)) & 1u) << e) | (((m1 >> (8 * e)) & 1u) << (4 + e));
        }
        smem[OFF_NAN + f4 * TILE + t] = uint8_t(nan);
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, row == -2);
        const bool any_nan = __any_sync(0xFFFFFFFFu, nan != 0);
        if (lane == 0) {
          reinterpret_cast<uint32_t*>(smem + OFF_BAD)[f4 * 4 + cw] = bad;
          reinterpret_cast<uint32_t*>(smem + OFF_FLAG)[f4 * 4 + cw] = (any_nan ? 1u : 0u) | (bad ? 2u : 0u);
          if (bad) atomicOr(status, DEV_BAD_INDEX);
        }
        uint32_t s2[8];
        scales(ks, s2);
        put(base + OFF_K + st * OP_BYTES, kc, s2);
        row = find(next_block, j + 1);
        load_k(row);
        fence_async_smem();
        warp_arrive(BAR(B_KFULL + st));
        if (kt >= 2) ok = wait_all(BAR(B_VEMPTY + st), ((kt >> 1) - 1) & 1);
        if (!ok) break;
        scales(vs, s2);
        put(base + OFF_V + st * OP_BYTES, vc, s2);
        load_v(row);
        next_block = entry(j + 2);
        fence_async_smem();
        warp_arrive(BAR(B_VFULL + st));
      }
      if (!ok) break;
    }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_SOFTMAX));
    const int x = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t col_s = tmem + lane_base + COL_S + 128u * uint32_t(x), col_o = tmem + lane_base + COL_O + 128u * uint32_t(x);
    const float vst = FMT == 1 ? __ldg(a.c.v_scale) : 1.0f;
    const float kst = FMT == 1 ? __ldg(a.c.k_scale) : 1.0f;
    float* s_cs = reinterpret_cast<float*>(smem + OFF_CS) + x * TILE + (warp & 3) * 32;  // of this warp's rows
    // this warp's 32 query rows of an item: binary16 with a power of two per row; eight
    // lanes per row, 16 channels each, all loads in flight at once
    const int tok4 = 4 / a.G, hd4 = 4 - tok4 * a.G;  // four rows further
    auto load_q = [&](const Item& it) {
      if ((x ? it.nb : it.na) == 0) return;
      const int part = lane & 7;
      uint4 v[8][2];
      int qr = x * TILE + (warp & 3) * 32 + (lane >> 3);
      int tok = (it.row0 + qr) / a.G, hd = it.row0 + qr - tok * a.G;
      const int tok0 = it.row0 / a.G, hd0 = it.row0 - tok0 * a.G;
#pragma unroll
      for (int p = 0; p < 8; p++) {
        // rows that are none take the item's first: nothing of them is written
        const int64_t t = it.q0 + (qr < it.rows ? tok : tok0);
        const uint16_t* src = a.q + t * a.q_stride + int64_t(it.h * a.G + (qr < it.rows ? hd : hd0)) * 128 + part * 16;
        v[p][0] = __ldg(reinterpret_cast<const uint4*>(src));
        v[p][1] = __ldg(reinterpret_cast<const uint4*>(src) + 1);
        qr += 4;
        tok += tok4;
        hd += hd4;
        if (hd >= a.G) {
          hd -= a.G;
          tok++;
        }
      }
#pragma unroll
      for (int p = 0; p < 8; p++) {
        const int lr = p * 4 + (lane >> 3), qr = (warp & 3) * 32 + lr;
        const uint32_t w[8] = {v[p][0].x, v[p][0].y, v[p][0].z, v[p][0].w, v[p][1].x, v[p][1].y, v[p][1].z, v[p][1].w};
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < 8; e++) mx = max(mx, hmax2(abs2(w[e])));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float2 sc = q_row_scale(mx);
        const uint32_t dst = base + OFF_Q + x * OP_BYTES + (part >> 2) * (OP_BYTES / 2) + qr * 128;
#pragma unroll
        for (int e = 0; e < 2; e++)
          st_shared_v4(dst + ((((part & 3) * 2 + e) ^ (qr & 7)) << 4), pack_f16(bf_lo(w[4 * e]) * sc.x, bf_hi(w[4 * e]) * sc.x),
                       pack_f16(bf_lo(w[4 * e + 1]) * sc.x, bf_hi(w[4 * e + 1]) * sc.x),
                       pack_f16(bf_lo(w[4 * e + 2]) * sc.x, bf_hi(w[4 * e + 2]) * sc.x),
                       pack_f16(bf_lo(w[4 * e + 3]) * sc.x, bf_hi(w[4 * e + 3]) * sc.x));
        // never 0: the score of a hidden key, -inf, is multiplied by it
        if (part == 0) s_cs[lr] = fmaxf(a.scale_log2 * kst * sc.y, 1.17549435e-38f);
      }
      fence_async_smem();
      warp_arrive(BAR(B_QFULL + x));
    };
    int st = 0, kt = 0;  // S products of this tile, tiles passed
    bool ok = true;
    Item it, next_it;
    int i = 0;
    bool more = take(i++, it, ok);
    if (more) load_q(it);
    for (; more; it = next_it) {
      const int n_x = x ? it.nb : it.na, nmax = max(it.na, it.nb);
      const int idx = x * TILE + row;
      const bool valid = idx < it.rows;
      const int tok = (it.row0 + idx) / a.G;
      const int klim = a.causal && valid ? it.kv - it.n + tok + 1 : it.kv;  // keys before it are visible
      // but not from kgap to kfrom - 1
      const int kgap = KIND == kWindow ? a.sinks : 0;
      const int kfrom = KIND == kWindow ? max(klim, 0) - a.window : KIND == kTail ? it.hi : 0;
      float m = -INFINITY, l = 0.0f;
      const float cs = n_x > 0 ? s_cs[lane] : 0.0f;
      uint32_t nan_blocks = 0;
      for (int n = 0; ok && n < 2 * n_x; n++) {
        const int j = n >> 1, h = n & 1;  // tile, half of its keys
        const uint32_t col = col_s + 64u * uint32_t(h);
        ok = wait_all(BAR(B_SFULL + 2 * x + h), uint32_t(st + j) & 1);
        if (!ok) break;
        tc_fence_after();
        float s[64];
#pragma unroll
        for (int c = 0; c < 2; c++) tmem_ld32(col + 32 * c, reinterpret_cast<uint32_t*>(s) + 32 * c);
        const int f4 = (kt + j) & 3;
        const volatile uint32_t* fl = reinterpret_cast<const volatile uint32_t*>(smem + OFF_FLAG) + f4 * 4 + 2 * h;
        const uint32_t flags = fl[0] | fl[1];
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; c++) reg_fence32(reinterpret_cast<uint32_t*>(s) + 32 * c);
        int kbase = (it.t0 + j) * TILE;
        if (kHides && kbase >= it.at) kbase += it.jump;
        kbase += 64 * h;
        if (kHides) {
          // a bit per key: a mask of bits costs little more than a select a key (comparisons two for each border)
          const uint64_t seen = below(klim - kbase) & (~below(kfrom - kbase) | below(kgap - kbase));
          if (__any_sync(0xFFFFFFFFu, ~seen != 0)) {
#pragma unroll
            for (int q = 0; q < 2; q++) {
              const uint32_t w = uint32_t(seen >> (32 * q));
#pragma unroll
              for (int e = 0; e < 32; e++)
                if (!((w >> e) & 1u)) s[32 * q + e] = -INFINITY;
            }
          }
        } else if (__any_sync(0xFFFFFFFFu, kbase + 64 > klim)) {
          const int lim = klim - kbase;
#pragma unroll
          for (int e = 0; e < 64; e++)
            if (e >= lim) s[e] = -INFINITY;
        }
        if (flags) {  // the same for the whole CTA
          const volatile uint32_t* bad = reinterpret_cast<const volatile uint32_t*>(smem + OFF_BAD) + f4 * 4 + 2 * h;
#pragma unroll
          for (int q = 0; q < 2; q++) {
            const uint32_t w = bad[q];
#pragma unroll
            for (int e = 0; e < 32; e++)
              if ((w >> e) & 1u) s[32 * q + e] = -INFINITY;
          }
          if (flags & 1u) {
            const volatile uint8_t* nb = smem + OFF_NAN + f4 * TILE + 64 * h;
            for (int e = 0; e < 64 && kbase + e < klim; e++)
              if (!kHides || kbase + e >= kfrom || kbase + e < kgap) nan_blocks |= nb[e];
          }
          __syncwarp();
        }
        float pm[2];  // two chains
#pragma unroll
        for (int q = 0; q < 2; q++) {
          pm[q] = fmaxf(s[32 * q], s[32 * q + 1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) pm[q] = fmax3(pm[q], s[32 * q + e], s[32 * q + e + 1]);
        }
        const float top = fmaxf(pm[0], pm[1]) * cs;
        float alpha = 1.0f;
        bool rescale = false;
        if (top > m + kLazy) {  // also from m = -inf on
          rescale = m != -INFINITY;
          alpha = rescale ? ex2(m - top) : 0.0f;
          m = top;
        }
        const float off = m == -INFINITY ? 0.0f : kOffset - m;
        uint32_t p[32];
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < 32; e++) {
          const float2 v = ffma2(make_float2(s[2 * e], s[2 * e + 1]), make_float2(cs, cs), make_float2(off, off));
          const float2 y = make_float2(ex2(v.x), ex2(v.y));
          sum = fadd2(sum, y);
          p[e] = pack_f16(y.x, y.y);
        }
        l = l * alpha + (sum.x + sum.y);
        // O_X is added to by the product of the half before; this half's waits for its P
        if (__any_sync(0xFFFFFFFFu, rescale)) {
          ok = wait_all(BAR(B_ODONE + 2 * x + (h ^ 1)), uint32_t(st + j - (h ^ 1)) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; c++) {
            uint32_t o[32];
            tmem_ld32(col_o + 32 * c, o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = fmul2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(alpha, alpha));
              o[e] = __float_as_uint(y.x);
              o[e + 1] = __float_as_uint(y.y);
            }
            tmem_st16(col_o + 32 * c, o);
            tmem_st16(col_o + 32 * c + 16, o + 16);
          }
        }
#pragma unroll
        for (int c = 0; c < 2; c++) tmem_st16(col + 16 * c, p + 16 * c);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(BAR(B_PFULL + 2 * x + h));
      }
      // the last S has been read, so the tile's queries may be replaced
      if (!ok) break;
      more = take(i++, next_it, ok);
      if (more) load_q(next_it);
      // the part's rows: O / l and lse, or a partial record
      if (ok && n_x > 0) ok = wait_all(BAR(B_ODONE + 2 * x + 1), uint32_t(st + n_x - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const float nanv = __uint_as_float(0x7FC00000u);
      const int hd = it.h * a.G + (it.row0 + idx) - tok * a.G;
      const int64_t out_row = int64_t(it.q0 + tok) * a.Hq + hd;
      // for the join: but not a request's whole rows without a prefix
      const bool keep = KIND == kPrefix || (KIND == kTail && (it.hi > 0 || it.slot >= 0));
      const float f = l == 0.0f ? 1.0f : vst / l;
      uint4* orow = reinterpret_cast<uint4*>(a.o + out_row * 128);
      float4* const record = reinterpret_cast<float4*>(it.slot < 0 ? a.rows_o + out_row * 128 : partials[it.slot].o[idx]);
#pragma unroll
      for (int c = 0; c < 4; c++) {
        float o[32];
        __syncwarp();
        if (n_x > 0) {
          tmem_ld32(col_o + 32 * c, reinterpret_cast<uint32_t*>(o));
          tmem_wait_ld();
          reg_fence32(reinterpret_cast<uint32_t*>(o));
        } else {
#pragma unroll
          for (int e = 0; e < 32; e++) o[e] = 0.0f;
        }
        if (nan_blocks) {
#pragma unroll
          for (int e = 0; e < 32; e++)
            if ((nan_blocks >> (2 * c + (e >> 4))) & 1u) o[e] = nanv;
        }
        if (valid && it.slot < 0 && !keep) {
#pragma unroll
          for (int e = 0; e < 4; e++)
            orow[4 * c + e] = make_uint4(pack_bf16(o[8 * e] * f, o[8 * e + 1] * f), pack_bf16(o[8 * e + 2] * f, o[8 * e + 3] * f),
                                         pack_bf16(o[8 * e + 4] * f, o[8 * e + 5] * f), pack_bf16(o[8 * e + 6] * f, o[8 * e + 7] * f));
        } else if (valid) {
          float4* const dst = record + 8 * c;
#pragma unroll
          for (int e = 0; e < 8; e++) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      tc_fence_before();
      if (valid) {
        if (it.slot >= 0) {
          partials[it.slot].m[idx] = m;
          partials[it.slot].l[idx] = l;
        } else if (keep) {
          a.rows_ml[out_row] = make_float2(m, l);
        } else {
          a.lse[int64_t(hd) * a.total_q + it.q0 + tok] = l == 0.0f ? -INFINITY : (m - kOffset + log2f(l)) * 0.6931471805599453f;
        }
      }
      if (keep && valid && it.t0 == 0) a.places[out_row] = make_uint2(blockIdx.x, kv_place(it.parts, idx, true, kHides && it.hi > 0));
      st += n_x;
      kt += nmax;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the item that begins in CTA blockIdx.x's run and ends behind
// it: one warp per row, four channels a lane, parts in the order of the keys.
template <int KIND, int FMT>
__global__ void __launch_bounds__(256) kv_prefill_join_kernel(KvAttnArgs a, const Header* headers, const Partial* partials) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the end of kv_prefill_kernel
  const Header hd = headers[blockIdx.x];
  if (hd.parts == 0) return;
  const int idx = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Request x = request_of<KIND>(a, hd.r);
  if (hd.row0 + idx >= x.n * a.G) return;
  auto part = [&](int i) -> const Partial& { return partials[2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)]; };
  float M = -INFINITY;
  for (int i = lane; i <= hd.parts; i += 32) M = fmaxf(M, part(i).m[idx]);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
  float L = 0.0f;
  float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 4
  for (int i = 0; i <= hd.parts; i++) {
    const Partial& p = part(i);
    const float m = p.m[idx];
    const float w = m == -INFINITY ? 1.0f : ex2(m - M);  // without keys l and O are 0, or NaN
    const float4 v = *reinterpret_cast<const float4*>(&p.o[idx][lane * 4]);
    L += w * p.l[idx];
    s.x += w * v.x;
    s.y += w * v.y;
    s.z += w * v.z;
    s.w += w * v.w;
  }
  const float vst = FMT == 1 ? __ldg(a.c.v_scale) : 1.0f;
  const int rr = hd.row0 + idx, tok = rr / a.G, head = hd.h * a.G + rr - tok * a.G;
  const int64_t row = int64_t(x.q0 + tok) * a.Hq + head;
  const float f = L == 0.0f ? 1.0f : vst / L;
  *reinterpret_cast<uint2*>(a.o + row * 128 + lane * 4) = make_uint2(pack_bf16(s.x * f, s.y * f), pack_bf16(s.z * f, s.w * f));
  if (lane == 0)
    a.lse[int64_t(head) * a.total_q + x.q0 + tok] =
        L == 0.0f ? -INFINITY : (M - kOffset + log2f(L)) * 0.6931471805599453f;
}

template <int KIND, int FMT>
cudaError_t launch(const KvAttnArgs& a, uint8_t* ws, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(kv_prefill_kernel<KIND, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  const int ctas = sm_count_current_device();
  if (ctas <= 0) return cudaErrorInvalidDevice;
  int64_t* line = reinterpret_cast<int64_t*>(ws);
  Header* headers = reinterpret_cast<Header*>(ws + line_bytes(a.R));
  Partial* partials = reinterpret_cast<Partial*>(ws + line_bytes(a.R) + header_bytes(ctas));
  e = launch_early(kv_prefill_kernel<KIND, FMT>, dim3(unsigned(ctas)), NTHREADS, SMEM_BYTES, st, a, static_cast<const int64_t*>(line), headers,
                   partials);
  if constexpr (kRecords<KIND>) return e;  // joined by kv_shared_join_kernel
  else
    return e != cudaSuccess ? e
                            : launch_early(kv_prefill_join_kernel<KIND, FMT>, dim3(unsigned(ctas), ROWS / 8), 256, 0, st, a,
                                           static_cast<const Header*>(headers), static_cast<const Partial*>(partials));
}

}  // namespace kvp

size_t kv_prefill_workspace(int R) {
  const int ctas = sm_count_current_device();
  return kvp::line_bytes(R) + kvp::header_bytes(ctas) + size_t(ctas) * 2 * sizeof(kvp::Partial);
}

uint8_t* kv_prefill_records(uint8_t* ws, int R) { return ws + kvp::line_bytes(R) + kvp::header_bytes(sm_count_current_device()); }

namespace {

template <int KIND>
cudaError_t launch_line(const KvAttnArgs& a, int64_t* line, bool after_attn, cudaStream_t st) {
  if (after_attn) return launch_early(kvp::kv_prefill_line_kernel<KIND>, dim3(1), 512, 0, st, a, line);
  kvp::kv_prefill_line_kernel<KIND><<<1, 512, 0, st>>>(a, line);
  return cudaGetLastError();
}

template <int KIND>
cudaError_t launch_kind(const KvAttnArgs& a, uint8_t* ws, cudaStream_t st) {
  return a.c.fmt == 0 ? kvp::launch<KIND, 0>(a, ws, st) : kvp::launch<KIND, 1>(a, ws, st);
}

}  // namespace

// The places of the requests on the line; `after_attn`: beside kv_attn_kernel, which is
// the launch before it.
cudaError_t launch_kv_prefill_line(int kind, const KvAttnArgs& a, uint8_t* ws, bool after_attn, cudaStream_t st) {
  int64_t* line = reinterpret_cast<int64_t*>(ws);
  switch (kind) {
    case kAll: return launch_line<kAll>(a, line, after_attn, st);
    case kWindow: return launch_line<kWindow>(a, line, after_attn, st);
    case kTail: return launch_line<kTail>(a, line, after_attn, st);
    default: return cudaErrorInvalidValue;  // the groups' line is kv_shared_plan_kernel's
  }
}

cudaError_t launch_kv_prefill(int kind, const KvAttnArgs& args, uint8_t* ws, cudaStream_t st) {
  KvAttnArgs a = args;
  // Every block for every head in one run, and the record that ends it.  Blocks: those of the requests that can have more
  // than split_rows rows, by the most tokens of one and by the tokens of all, a part of a block more for each.  The second
  // counts where max_q is a capacity: 63 requests of one token beside one of 60 take 47 us with max_q = 60 as with 2^30 (282
  // by the first alone).
  const int64_t rows = a.total_q * a.G, most_q = a.max_q < a.total_q ? a.max_q : a.total_q;
  const int64_t above = rows / (int64_t(a.split_rows) + 1), requests = a.R < above ? a.R : above;
  const int64_t by_one = requests * ((most_q * a.G + kvp::ROWS - 1) / kvp::ROWS), by_all = rows / kvp::ROWS + requests;
  const int64_t items = (by_one < by_all ? by_one : by_all) * a.c.H + 1;
  a.item_loops = int(ceil(cbrt(double(items)))) + 1;
  a.item_most = int(items < (int64_t(1) << 30) ? items : int64_t(1) << 30);
  switch (kind) {
    case kAll: return launch_kind<kAll>(a, ws, st);
    case kWindow: return launch_kind<kWindow>(a, ws, st);
    case kPrefix: return launch_kind<kPrefix>(a, ws, st);
    default: return launch_kind<kTail>(a, ws, st);
  }
}

unsigned read_status_kv_prefill(cudaStream_t st) {
  unsigned v = 0, z = 0;
  cudaMemcpyFromSymbolAsync(&v, g_status_kv_prefill, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  cudaMemcpyToSymbolAsync(g_status_kv_prefill, &z, sizeof(z), 0, cudaMemcpyHostToDevice, st);
  cudaStreamSynchronize(st);
  return v;
}

}  // namespace mxfa
