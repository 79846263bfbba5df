// hq_prompt.cu -- attention over packed prompts (include/hq_prompt.h).
//
// A tile is 128 query rows of one (sequence, query head).  A block works on two
// tiles that read the same K and V: two heads of a group over the same
// rows, or, for the last head of an odd group, two neighbouring tiles.  K and V come
// 128 rows at a time through a ring of TMA copies; per tile and 128 keys
//   S = Q K^T        tensor cores, operands in shared memory, S in tensor memory
//   P = 2^(c (S - m)), l += P's row sums, m the row's reference    a thread a row
//   O += P V         P from tensor memory (in S's place), V from shared memory
// Warps 0 .. 3 and 4 .. 7 are the two tiles' rows, warp 8 asks for copies, warp 9 for
// products, which run while one tile's softmax overlaps the other tile's products.  The
// reference is taken from the maximum of a row's first scores and moves only when a weight
// passes 2^60 (bf16; 2^5 in fp16) times that score's, so O, which then has to be read and scaled, is left
// alone nearly always (bf16) or mostly (fp16).
//
// 16384 tokens, 32 heads on 8, bf16: 1.40 ms, 1.57 PFLOP/s, one call a graph's replay, 83% of the rate measured for
// cuBLAS in a burst and 94% of what it sustains; call after call 1.47 to 1.50 ms, 1.48 PFLOP/s.  128 keys take a block 3000 to
// 3200 cycles: a tile's softmax 1300 (450 instructions a warp; exponentials alone 512), both products 1330, of 1024 at
// the pipe's full rate, and the waits between; the other tile is half a turn behind.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "hq_kv4_io.cuh"
#include "hq_launch.cuh"
#include "hq_prompt.h"
#include "hq_score.cuh"
#include "hq_umma.cuh"

namespace hq {

namespace {

constexpr int kKeys = 128;                       // keys of a block of K and V
constexpr int kThreads = 384;                    // three groups of four warps, the last two warps without work
// Registers: 168 a thread at launch; a row takes 208, its weights among them, copies and products 88.
constexpr int kLaunchRegs = 168, kRowRegs = 208, kOtherRegs = 88;
static_assert(2 * kRowRegs + kOtherRegs <= 3 * kLaunchRegs, "no more than the block was launched with");
constexpr int kStages = 4;                       // blocks of K or V in the ring
constexpr int kTileBytes = kPromptRows * kTile * 2;          // 32 KB: two halves of 64 dimensions
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kOutBytes = 32 * 128;              // of a warp, on the way out: 32 rows of 64 dimensions
constexpr int kSmem = (2 + kStages) * kTileBytes + 8 * kOutBytes + 1024;     // 1024: alignment
constexpr uint32_t kIdesc = umma_idesc_f16(kPromptRows, kKeys);
// log2 of the weight that a reference gives the score it is taken from, and of the largest weight that does not
// move it.  In fp16 weights keep their 11 bits down to 2^-14, so the row's largest weight is held at 2^10 to 2^15: those
// of 2^-24 of it and more are rounded by 2^-11 of themselves, smaller ones by up to 2^-35 of the largest.  (Prompt
// of 16384 tokens whose scores climb by some tens, fp16, us: 2024; 1984 from 2^8 on, 1947 from 2^6, 1822 from 1, 1738 with
// 2^-6 to 2^14, where one heavy key of small value over 16384 others left 9% of the outputs' size as an error.)
// In bf16 weights keep their bits whatever their size; what has to fit fp32 are the sums of weights and values: 2^30
// above the reference they do while V's magnitudes come to less than 2^97, 2^-30 below it they keep parts of 2^-96 of an
// output.  (The same prompt in bf16: 1402; 1472 with 2^-20 to 2^20, 1554 with 2^-15 to 2^15, 1959 with 1 to 2^8; 1399 with
// 1 to 2^60, where values from 2^68 on came out infinite.)
template <int KIND> constexpr float kFirst = KIND == HQ_T_BF16 ? -30.0f : 10.0f;
template <int KIND> constexpr float kMost = KIND == HQ_T_BF16 ? 30.0f : 15.0f;

// What a block does next: two tiles (A, B) that share K and V.
struct Item {
  int q[2];                                      // first row
  int n[2];                                      // rows, 0: no tile
  int seen[2];                                   // keys that the first row sees (may be below 1)
  int head[2];                                   // in its group
  int k, keys;                                   // the sequence's first K row, and their number
  int pad[2];
};
static_assert(sizeof(Item) == 48, "three 16-byte loads");

// What a launch goes by, made on the device from the lengths.  Items are (unit of the list, KV head).
// They are dealt out whole, or, where that leaves some blocks with far more than others, the
// batch, items laid end to end as their blocks of keys behind kItemCost, is cut into pieces of
// `per`, one a block of the grid; a tile that several share is then joined from their sums.
constexpr int kMostBlocks = 160;                 // of the grid
constexpr int kItemCost = 3;                     // what it takes to begin and end an item, in blocks of keys
constexpr int kSplitUnits = 8 * kMostBlocks;     // most items of a batch that may be cut
struct Plan {
  int count;                                     // units
  int per;                                       // 0: items are dealt out whole
  int pad[2];
  int4 begin[kMostBlocks];                       // unit, KV head and place in the item that a piece begins at; its length
  int4 join[kMostBlocks];                        // a tile's unit and KV head; the blocks of keys that this piece has of it,
};                                               // and how many pieces follow (0: nothing begins here that others end)
// Sums of a piece that ends or begins inside an item: tiles A and B, [32 groups of 4 dimensions][128 rows].
struct Part {
  float4 sums[2][kTile / 4][kPromptRows];
  float2 stat[2][kPromptRows];                   // reference, sum of weights
};
// A piece has room for the item that it begins inside of, and for the one that it ends inside of.  The blocks of keys of
// all items, with their costs, are added up in 32 bits.
__host__ __device__ __forceinline__ bool may_split(int64_t units, int n_kv, int64_t n_k_tokens) {
  return units * n_kv <= kSplitUnits && n_k_tokens > 16 * kKeys &&
         units * n_kv * (n_k_tokens / kKeys + 1 + kItemCost) <= INT_MAX;
}

// Where sequence b's rows begin and end, held to [0, n].
__device__ __forceinline__ int2 rows_of(const int32_t *starts, int b, int n, bool *bad) {
  const int s = starts[b], e = starts[b + 1];
  const int lo = min(max(s, 0), n), hi = min(max(e, 0), n);
  *bad = *bad || lo != s || hi != e || hi < lo;
  return make_int2(lo, max(lo, hi));
}
__device__ __forceinline__ int blocks_of(int seen, int n) {     // that the last of n rows sees
  return n == 0 ? 0 : (max(0, seen + n - 1) + kKeys - 1) / kKeys;
}

__device__ __forceinline__ int tiles_of(int2 rows) { return (rows.y - rows.x + kPromptRows - 1) / kPromptRows; }
// Units of a sequence: pairs of heads, tile by tile, then the last head of an odd group, two tiles at a time.
__device__ __forceinline__ int units_of(int tiles, int G) { return G / 2 * tiles + (G & 1) * ((tiles + 1) / 2); }
__device__ __forceinline__ Item item_of(int2 qr, int2 kr, int G, int unit) {
  const int n = qr.y - qr.x, keys = kr.y - kr.x, tiles = tiles_of(qr), paired = G / 2 * tiles;
  int t0, t1, head;
  if (unit < paired) {
    t0 = t1 = unit / (G / 2);
    head = 2 * (unit - t0 * (G / 2));
  } else {
    t0 = 2 * (unit - paired);
    t1 = t0 + 1;
    head = G - 1;
  }
  Item x;
  x.q[0] = qr.x + t0 * kPromptRows;
  x.q[1] = qr.x + t1 * kPromptRows;
  x.n[0] = min(kPromptRows, n - t0 * kPromptRows);
  x.n[1] = max(0, min(kPromptRows, n - t1 * kPromptRows));
  x.seen[0] = keys - n + t0 * kPromptRows + 1;
  x.seen[1] = keys - n + t1 * kPromptRows + 1;
  x.head[0] = head;
  x.head[1] = unit < paired ? head + 1 : head;
  x.k = kr.x;
  x.keys = keys;
  x.pad[0] = x.pad[1] = 0;
  return x;
}
__device__ __forceinline__ int item_blocks(const Item &x) {
  return max(blocks_of(x.seen[0], x.n[0]), blocks_of(x.seen[1], x.n[1]));
}
// The batch's unit of a number, found by a warp from the lengths; false: there is none.
__device__ bool unit_of(const PromptArgs &a, int unit, Item &x) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < a.n_seqs; b0 += 32) {
    const int b = b0 + lane;
    bool bad = false;
    int2 qr = make_int2(0, 0), kr = qr;
    if (b < a.n_seqs) {
      qr = rows_of(a.starts, b, a.n_tokens, &bad);
      kr = rows_of(a.k_starts, b, a.n_k_tokens, &bad);
    }
    const int mine = units_of(tiles_of(qr), a.G);
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    if (unit < total) {
      const int from = __popc(__ballot_sync(0xffffffffu, incl <= unit));       // sequences that end before
      unit -= __shfl_sync(0xffffffffu, incl - mine, from);
      qr = make_int2(__shfl_sync(0xffffffffu, qr.x, from), __shfl_sync(0xffffffffu, qr.y, from));
      kr = make_int2(__shfl_sync(0xffffffffu, kr.x, from), __shfl_sync(0xffffffffu, kr.y, from));
      x = item_of(qr, kr, a.G, unit);
      return true;
    }
    unit -= total;
  }
  return false;
}
// Returns the units of the sequences that it looked at.
__device__ int64_t check_starts(const PromptArgs &a, int first, int step) {
  bool bad = false;
  int64_t units = 0;
  for (int b = first; b < a.n_seqs; b += step) {
    units += units_of(tiles_of(rows_of(a.starts, b, a.n_tokens, &bad)), a.G);
    rows_of(a.k_starts, b, a.n_k_tokens, &bad);
  }
  if (bad) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
  return units;
}

// The list of units, longest first (a counting sort by blocks of keys): a unit
// times the KV heads makes that many items.  A warp a sequence, a lane a unit.  Units that
// the sort does not tell apart come as their warps do where items are dealt out whole.  Where they
// may be cut, the place in the list decides at which key, and so the order of a row's sums: there such
// units keep the batch's order, ranked by one warp, 32 at a time.  Where
// there are no more items than blocks of the grid, those find them by themselves
// (prompt of 77 tokens, 32 heads: 8 us, 12 with a list).
constexpr int kPrepThreads = 1024, kBuckets = 1024;
__global__ void __launch_bounds__(kPrepThreads)
    prompt_prep_kernel(PromptArgs a, Plan *plan, Item *list, int room, int grid, int split) {
  __shared__ int s_at[kBuckets];
  __shared__ int s_warp[32];
  __shared__ int s_end[kSplitUnits + 1];         // blocks of keys up to a unit's end
  __shared__ int s_first[kSplitUnits];           // a sequence's first unit, in the batch's order
  __shared__ uint16_t s_rank[kSplitUnits];       // a unit's bucket, then its place in the list
  __shared__ int s_most;
  __shared__ unsigned long long s_units;
  follow_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  s_at[tid] = 0;
  if (tid == 0) {
    s_most = 0;
    s_units = 0;
  }
  __syncthreads();
  const int64_t own = check_starts(a, tid, kPrepThreads);
  if (own > 0) atomicAdd(&s_units, (unsigned long long)own);
  __syncthreads();
  if (s_units > (unsigned long long)room) {      // starts that descend name rows many times over: no list holds them
    if (tid == 0) plan->count = plan->per = 0;
    return;
  }
  if (split) {                                   // no more sequences than units: a thread two of them
    static_assert(kSplitUnits <= 2 * kPrepThreads, "a thread two sequences or units");
    int u[2] = {0, 0};
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (2 * tid + k < a.n_seqs) u[k] = units_of(tiles_of(rows_of(a.starts, 2 * tid + k, a.n_tokens, &bad)), a.G);
    int incl = u[0] + u[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int first = incl - u[0] - u[1];
    for (int w = 0; w < warp; ++w) first += s_warp[w];
    if (2 * tid < a.n_seqs) s_first[2 * tid] = first;
    if (2 * tid + 1 < a.n_seqs) s_first[2 * tid + 1] = first + u[0];
    __syncthreads();
  }
  const auto walk = [&](auto &&put) {
    for (int b = warp; b < a.n_seqs; b += kPrepThreads / 32) {
      bool bad = false;
      const int2 qr = rows_of(a.starts, b, a.n_tokens, &bad), kr = rows_of(a.k_starts, b, a.n_k_tokens, &bad);
      const int units = units_of(tiles_of(qr), a.G);
      for (int u = lane; u < units; u += 32) {
        const Item x = item_of(qr, kr, a.G, u);
        put(kBuckets - 1 - min(kBuckets - 1, item_blocks(x)), x, split ? s_first[b] + u : 0);
      }
    }
  };
  walk([&](int bucket, const Item &, int number) {
    atomicAdd(&s_at[bucket], 1);
    if (split) s_rank[number] = (uint16_t)bucket;
  });
  __syncthreads();
  const int mine = s_at[tid];
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  s_at[tid] = before + incl - mine;
  if (tid == kBuckets - 1) s_end[0] = before + incl;
  __syncthreads();
  const int count = s_end[0];
  if (split && warp == 0) {
    for (int n0 = 0; n0 < count; n0 += 32) {
      const bool is = n0 + lane < count;
      const int bucket = is ? s_rank[n0 + lane] : kBuckets;
      const uint32_t same = __match_any_sync(0xffffffffu, bucket);
      const int from = is ? s_at[bucket] : 0;
      __syncwarp();
      if (is) s_rank[n0 + lane] = (uint16_t)(from + __popc(same & ((1u << lane) - 1u)));
      if (is && same >> lane == 1u) s_at[bucket] = from + __popc(same);     // the last of them
      __syncwarp();
    }
  }
  __syncthreads();
  walk([&](int bucket, const Item &x, int number) {
    const int at = split ? s_rank[number] : atomicAdd(&s_at[bucket], 1);
    list[at] = x;
    if (split) s_end[at + 1] = item_blocks(x);
  });
  if (tid == 0) plan->count = count;
  if (!split) {
    if (tid == 0) plan->per = 0;
    return;
  }
  // where the units end, rows that see nothing counted as one block: a thread two of them
  if (tid == 0) s_end[0] = 0;
  __syncthreads();
  int e[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (2 * tid + k < count) e[k] = kItemCost + max(1, s_end[2 * tid + k + 1]) + (k == 1 ? e[0] : 0);
  int sum = max(e[0], e[1]);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  int base = sum - max(e[0], e[1]);
  for (int w = 0; w < warp; ++w) base += s_warp[w];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (2 * tid + k < count) s_end[2 * tid + k + 1] = base + e[k];
  __syncthreads();
  const int64_t all = (int64_t)s_end[count] * a.n_kv;
  // The longest share when items are dealt out whole, and in pieces: there about 16 more for the sums that are
  // written and joined.
  const int items = count * a.n_kv;
  if (tid < grid) {
    int mine = 0;
    for (int round = 0; round * grid < items; ++round) {
      const int id = round * grid + ((round & 1) ? grid - 1 - tid : tid);
      if (id < items) mine += s_end[id / a.n_kv + 1] - s_end[id / a.n_kv];
    }
    atomicMax(&s_most, mine);
  }
  __syncthreads();
  const int64_t per = (all + grid - 1) / grid;
  const bool cut = per + 16 < s_most;
  if (tid == 0) plan->per = cut ? (int)per : 0;
  if (!cut || tid >= grid) return;
  const auto find = [&](int64_t pos) {           // unit, KV head, place in the item and its span, of a place of the batch
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)s_end[mid + 1] * a.n_kv > pos) hi = mid;
      else lo = mid + 1;
    }
    const int span = s_end[lo + 1] - s_end[lo], rest = (int)(pos - (int64_t)s_end[lo] * a.n_kv);
    return make_int4(lo, rest / span, rest % span, span);
  };
  const int64_t from = min(all, tid * per), to = min(all, from + per);
  int4 begin = make_int4(0, 0, 0, 0), join = make_int4(0, 0, 0, 0);
  if (from < to) {
    const int4 f = find(from);
    begin = make_int4(f.x, f.y, f.z, (int)(to - from));
    if (to < all) {
      const int4 t = find(to);                   // inside an item whose first block of keys is in this piece?
      if (t.z > kItemCost && to - t.z + kItemCost >= from)
        join = make_int4(t.x, t.y, t.z - kItemCost, (int)((t.w - t.z + per - 1) / per));
    }
  }
  plan->begin[tid] = begin;
  plan->join[tid] = join;
}

struct PromptMaps {
  CUtensorMap q, k, v;
};

struct Bars {
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t full[kStages], empty[kStages];
  uint64_t patch;
};

// What scores are multiplied by to be exponents of 2.  Not 0: -inf stays -inf, and no finite score is anything.
template <bool CAP>
__device__ __forceinline__ float factor_of(const PromptArgs &a) {
  const float c = fabsf(__fmul_rn(a.scale, kLog2e));
  return CAP ? 1.0f : c == 0.0f ? 0x1p-149f : c;
}
__device__ __forceinline__ float lse_of(float m, float l, float c) {
  return l == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(__fmul_rn(m, c), log2f(l)), kLn2);
}

template <int KIND>
__device__ __forceinline__ uint32_t pack2(uint64_t p) {
  float lo, hi;
  upk2(p, lo, hi);
  return round_pair<KIND>(lo, hi);
}

// What a block of the grid does, item after item; the warps that walk do so alike.
struct Walk {
  const Plan *plan;
  const Item *list;
  int items, n_kv, round;
  int unit, head, at, left;                      // of a piece; left < 0: whole items
  Item ahead;
  __device__ __forceinline__ Walk(const PromptArgs &a, const Plan *p, const Item *l) : plan(p), list(l), n_kv(a.n_kv), round(0), left(-1) {
    if (plan == nullptr) {                       // one item at most
      items = unit_of(a, (int)(blockIdx.x / (uint32_t)n_kv), ahead) ? (int)blockIdx.x + 1 : 0;
      return;
    }
    items = plan->count * n_kv;
    if (plan->per != 0) {
      const int4 b = plan->begin[blockIdx.x];
      unit = b.x;
      head = b.y;
      at = b.z;
      left = b.w;
    } else {
      ask();
    }
  }
  // the list is dealt out back and forth, so that no block gets the longest of every round
  __device__ __forceinline__ int id() const {
    return round * (int)gridDim.x + ((round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
  }
  __device__ __forceinline__ void ask() {        // the next item's description, before it is needed
    if (id() < items) ahead = list[(uint32_t)id() / (uint32_t)n_kv];
  }
  // The next item, its KV head, and its blocks of keys lo .. hi - 1 that are this block's.
  __device__ __forceinline__ bool next(Item &x, int &h, int &lo, int &hi) {
    if (left < 0) {
      const int i = id();                        // only the last round has no item for some
      if (i >= items) return false;
      x = ahead;
      h = (int)((uint32_t)i % (uint32_t)n_kv);
      lo = 0;
      hi = INT_MAX;
      ++round;
      ask();
      return true;
    }
    do {                                         // a piece may begin or end in an item's cost
      if (left == 0) return false;
      x = list[unit];
      h = head;
      const int span = kItemCost + max(1, item_blocks(x));
      const int end = min(span, at + left);
      lo = max(0, at - kItemCost);
      hi = max(0, end - kItemCost);
      left -= end - at;
      at = end;
      if (at == span) {
        at = 0;
        if (++head == n_kv) {
          head = 0;
          ++unit;
        }
      }
    } while (hi <= lo);
    return true;
  }
};

template <int KIND, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ PromptMaps maps, PromptArgs a, const Plan *plan, const Item *list, Part *parts) {
  extern __shared__ unsigned char s_raw[];
  __shared__ Bars s_bar;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t ring = base + 2 * kTileBytes;
  volatile int *const abort = &s_abort;
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    if (lane == 0) {
      tma_prefetch_map(&maps.q);
      tma_prefetch_map(&maps.k);
      tma_prefetch_map(&maps.v);
    }
  }
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_bar.q_full[i], 1);
      mbar_init(&s_bar.q_empty[i], 1);
      mbar_init(&s_bar.s_full[i], 1);
      mbar_init(&s_bar.p_full[i], 4);
      mbar_init(&s_bar.o_full[i], 1);
      mbar_init(&s_bar.o_empty[i], 4);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s_bar.full[i], 1);
      mbar_init(&s_bar.empty[i], 1);
    }
    mbar_init(&s_bar.patch, 1);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  follow_launch();
  const uint32_t tmem = s_tmem;
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // -------------------------------------------------------------- copies
      const bool leader = elect_one();
      uint32_t stage = 0, turn = 0, used[2] = {0, 0}, patches = 0;
      const auto ask = [&](const CUtensorMap &map, uint32_t dst, uint64_t *bar, int head, int row) {
        if (!leader) return;
        mbar_expect(bar, kTileBytes);
        tma_load3(dst, &map, bar, 0, head, row);
        tma_load3(dst + kHalfBytes, &map, bar, 64, head, row);
      };
      Walk walk(a, plan, list);
      Item x;
      int h, lo, hi;
      while (walk.next(x, h, lo, hi)) {
        const int nb[2] = {min(hi, blocks_of(x.seen[0], x.n[0])), min(hi, blocks_of(x.seen[1], x.n[1]))};
        const int most = max(nb[0], nb[1]);
        const auto query = [&](int i) {
          if (nb[i] <= lo) return;
          wait(&s_bar.q_empty[i], used[i] + 1, abort);
          ask(maps.q, base + i * kTileBytes, &s_bar.q_full[i], h * a.G + x.head[i], x.q[i]);
          ++used[i];
        };
        query(0);
        for (int j = 2 * lo; j < 2 * most; ++j) {
          const int row = (j >> 1) * kKeys, left = x.keys - row;
          const uint32_t dst = ring + stage * kTileBytes;
          const bool is_v = j & 1, partial = is_v && left < kKeys;
          wait(&s_bar.empty[stage], turn + 1, abort);
          ask(is_v ? maps.v : maps.k, dst, partial ? &s_bar.patch : &s_bar.full[stage], h, x.k + row);
          if (partial) {
            // rows behind the sequence's end are another's, or nobody's: zeros, as 0 times what is there may be NaN
            wait(&s_bar.patch, patches++, abort);
            for (int c = left * 8 + lane; c < kKeys * 8; c += 32)
#pragma unroll
              for (int half = 0; half < 2; ++half)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + half * kHalfBytes + c * 16), "r"(0)
                             : "memory");
            fence_async_smem();
            __syncwarp();
            if (leader) mbar_arrive(&s_bar.full[stage]);
          }
          if (++stage == kStages) {
            stage = 0;
            ++turn;
          }
          if (j == 2 * lo) query(1);
        }
      }
      if (*abort) {                              // copies in flight end before the block does
        for (int i = 0; i < 2; ++i)
          if (used[i] > 0) mbar_wait(&s_bar.q_full[i], (used[i] - 1) & 1u, 1u << 16);
        for (int i = 0; i < kStages; ++i) {
          const uint32_t t = i < (int)stage ? turn : turn - 1;
          if (i < (int)stage || turn > 0) mbar_wait(&s_bar.full[i], t & 1u, 1u << 16);
        }
      }
    } else if (warp == 9) {
      // -------------------------------------------------------------- products
      // The warp runs as one, its values uniform, with a leader's instructions in between.
      const bool leader = elect_one();
      constexpr uint32_t kind = kIdesc | (KIND == HQ_T_BF16 ? kUmmaBf16 : 0u);
      const uint32_t qk = kind | (a.scale < 0.0f ? kUmmaNegateA : 0u), pv = kind | kUmmaBMnMajor;
      uint32_t stage = 0, turn = 0, used[2] = {0, 0}, steps[2] = {0, 0};
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), base_u = __shfl_sync(0xffffffffu, base, 0);
      const uint32_t ring_u = base_u + 2 * kTileBytes;
      const auto next_stage = [&] {
        if (++stage == kStages) {
          stage = 0;
          ++turn;
        }
      };
      const auto commit = [&](uint64_t *bar) {
        if (leader) umma_commit(bar);
      };
      const auto scores = [&](int i, uint32_t at) {              // S of tile i with the K of stage `at`
        const uint64_t q = umma_desc_sw128(base_u + i * kTileBytes, 16);
        const uint64_t k = umma_desc_sw128(ring_u + at * kTileBytes, 16);
        if (leader) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t off = ((e >> 2) * kHalfBytes + (e & 3) * 32) >> 4;
            umma_f16(tm + i * 128, q + off, k + off, qk, e > 0);
          }
          umma_commit(&s_bar.s_full[i]);
        }
      };
      Walk walk(a, plan, list);
      Item x;
      int h, from, to;
      while (walk.next(x, h, from, to)) {
        const int nb[2] = {__shfl_sync(0xffffffffu, min(to, blocks_of(x.seen[0], x.n[0])), 0),
                           __shfl_sync(0xffffffffu, min(to, blocks_of(x.seen[1], x.n[1])), 0)};
        const int most = max(nb[0], nb[1]), lo = __shfl_sync(0xffffffffu, from, 0);
        if (most <= lo) continue;
        wait(&s_bar.full[stage], turn, abort);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (nb[i] <= lo) continue;
          wait(&s_bar.q_full[i], used[i], abort);
          tc_fence_after();
          scores(i, stage);
          if (nb[i] == lo + 1) commit(&s_bar.q_empty[i]);
        }
        commit(&s_bar.empty[stage]);
        next_stage();
        for (int j = lo; j < most; ++j) {
          const uint32_t v_stage = stage;
          wait(&s_bar.full[stage], turn, abort);
          next_stage();
          bool k_there = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (j >= nb[i]) continue;
            if (j == lo) wait(&s_bar.o_empty[i], used[i] + 1, abort);
            wait(&s_bar.p_full[i], steps[i]++, abort);
            tc_fence_after();
            const uint64_t v = umma_desc_sw128(ring_u + v_stage * kTileBytes, kHalfBytes);
            if (leader) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                umma_f16_ts(tm + 256 + i * 128, tm + i * 128 + 8 * e, v + ((e * 2048) >> 4), pv, j > lo || e > 0);
            }
            if (j + 1 < nb[i]) {
              if (!k_there) wait(&s_bar.full[stage], turn, abort);
              k_there = true;
              scores(i, stage);
              if (j + 2 == nb[i]) commit(&s_bar.q_empty[i]);
            } else {
              commit(&s_bar.o_full[i]);
            }
          }
          commit(&s_bar.empty[v_stage]);
          if (j + 1 < most) {
            commit(&s_bar.empty[stage]);
            next_stage();
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) used[i] += nb[i] > lo;
      }
      if (*abort) {                              // products in flight end before the block does
        commit(&s_bar.patch);
        for (uint32_t p = 0; p < 2; ++p) mbar_wait(&s_bar.patch, p, 1u << 16);
      }
    } else if (warp == 10 && plan == nullptr && blockIdx.x == 0) {
      check_starts(a, lane, 32);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    // ---------------------------------------------------------------- rows
    const int i = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_s = tmem + i * 128 + lanes, t_o = tmem + 256 + i * 128 + lanes;
    const uint32_t staged = ring + kStages * kTileBytes + warp * kOutBytes;
    const float c = factor_of<CAP>(a);
    const float scale = fabsf(a.scale), by_cap = CAP ? __fdiv_rn(1.0f, a.cap) : 0.0f, cap_l2 = __fmul_rn(a.cap, kLog2e);
    constexpr float most_weight = kMost<KIND>;
    // The reference that gives a score the weight 2^kFirst; 1 from 2^24 on, where scores have no place for it.
    const float margin = c > 0x1p-60f ? __fdiv_rn(-kFirst<KIND>, c) : 0.0f;
    const auto ref_of = [&](float score) {
      return fabsf(__fmul_rn(score, c)) < 0x1p24f ? __fadd_rn(score, margin) : score;
    };
    const float to_y = fminf(__fmul_rn(scale, by_cap), 3e38f), to_l2 = __fmul_rn(scale, kLog2e);
    uint32_t steps = 0, used = 0;
    Walk walk(a, plan, list);
    Item x;
    int h, lo, hi;
    while (walk.next(x, h, lo, hi)) {
      const int n = i == 0 ? x.n[0] : x.n[1], seen = i == 0 ? x.seen[0] : x.seen[1], all = blocks_of(seen, n);
      const int nb = min(hi, all);
      const bool mine = row < n;                 // the tile has this row; others have no say in what it does
      if (lo > 0 && nb <= lo) continue;          // the other tile's blocks alone
      const int64_t at = (int64_t)((i == 0 ? x.q[0] : x.q[1]) + row) * a.Hq + h * a.G + (i == 0 ? x.head[0] : x.head[1]);
      float m = -INFINITY;                       // the row's reference, a score as the products give it
      uint64_t l2 = 0;                           // two sums of weights
      for (int j = lo; j < nb; ++j) {
        wait(&s_bar.s_full[i], steps++, abort);
        tc_fence_after();
        const int lim = seen + row - j * kKeys;  // keys of this block that the row sees
        const bool masked = seen - j * kKeys < kKeys;            // not all rows see all of them
        // 32 scores as they enter the softmax
        const auto take = [&](uint32_t s[32], int k0) {
          const int left = lim - k0;
          const uint32_t sees = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
          const auto hide = [&](uint32_t with) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(sees & (1u << k))) s[k] = with;
          };
          if (CAP) {
            if (masked) hide(0u);                // what is not seen has no say in what follows
            cap32(s, mine, scale, to_y, to_l2, by_cap, cap_l2);
          }
          if (masked) hide(0xFF800000u);
        };
        const auto top_of = [&](const uint32_t s[32], float top[2]) {
#pragma unroll
          for (int k = 0; k < 32; k += 4)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              top[e] = max3(top[e], __uint_as_float(s[k + 2 * e]), __uint_as_float(s[k + 2 * e + 1]));
        };
        uint32_t w[kKeys / 2];                   // weights, two a word
        uint64_t sum[2];
        // Moves the reference for rows whose scores' maximum passed it by too much, and scales what there is.
        const auto move = [&](float most, bool far) {
          const float now = far ? ref_of(most) : m;
          if (j > lo) {
            const float by = m == now ? 1.0f : m == -INFINITY ? 0.0f : ex2(__fmul_rn(__fsub_rn(m, now), c));
            l2 = mul2(l2, pk2(by, by));
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {        // this block's scores are there, so all products before them are
              uint32_t o[32];
              tmem_ask32(t_o + 32 * k, o);
              tmem_wait32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), by));
              tmem_st32(t_o + 32 * k, o);
            }
          }
          m = now;
        };
        bool again = false, less = false;        // the weights once more; the scores have the reference taken off
        if (CAP) {                               // capped once, in their place, and the maximum known before the weights
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            uint32_t s[32];
            tmem_ask32(t_s + 32 * k, s);
            tmem_wait32(s);
            take(s, 32 * k);
            top_of(s, top);
            tmem_st32(t_s + 32 * k, s);
          }
          tmem_wait_st();
          const float most = fmaxf(top[0], top[1]);
          const bool far = j == lo || __fsub_rn(most, m) > most_weight;
          if (__any_sync(0xffffffffu, mine && far)) move(most, far);
          again = true;
        }
        while (true) {
          // Weights and their sums against the reference, and the scores' maximum beside them: 32 scores
          // on their way while the 32 before them are worked on.  An item's first reference is the maximum of
          // its first 32 scores.
          float top[2] = {-INFINITY, -INFINITY};
          uint64_t m2, mc2;
          const uint64_t c2 = pk2(c, c);
          uint32_t s[2][32];
          sum[0] = sum[1] = 0;
          tmem_ask32(t_s, s[0]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t *const now = s[k & 1];
            tmem_wait32(now);
            if (k < 3) tmem_ask32(t_s + 32 * (k + 1), s[(k + 1) & 1]);
            if (!CAP && !less) take(now, 32 * k);
            if (!CAP) top_of(now, top);
            if (k == 0) {
              if (j == lo && !again) m = ref_of(fmaxf(top[0], top[1]));
              const float from = less || m == -INFINITY ? 0.0f : m, mc = __fmul_rn(from, c);
              m2 = pk2(from, from);
              mc2 = pk2(-mc, -mc);
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              const uint64_t z = pk2(__uint_as_float(now[e]), __uint_as_float(now[e + 1]));
              upk2(CAP ? sub2(z, m2) : fma2(z, c2, mc2), x0, x1);
              const uint64_t p = pk2(ex2(x0), ex2(x1));
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], p);
              w[16 * k + (e >> 1)] = pack2<KIND>(p);
            }
          }
          if (again) break;
          // Once more where a weight passed the reference by too much; and where c m is so large that its
          // rounding, the same for the whole row, matters by itself: there m is taken off the scores first.
          const bool far = __fmul_rn(__fsub_rn(fmaxf(top[0], top[1]), m), c) > most_weight;
          const float size = fabsf(__fmul_rn(m, c));
          const bool large = size >= 0x1p20f && size < INFINITY;
          if (!__any_sync(0xffffffffu, mine && (far || large))) break;
          again = true;
          less = __any_sync(0xffffffffu, mine && large);
          move(fmaxf(top[0], top[1]), far);
          if (less) {
            const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              uint32_t o[32];
              tmem_ask32(t_s + 32 * k, o);
              tmem_wait32(o);
              take(o, 32 * k);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fsub_rn(__uint_as_float(o[e]), from));
              tmem_st32(t_s + 32 * k, o);
            }
            tmem_wait_st();
          }
        }
        l2 = add2(l2, add2(sum[0], sum[1]));
        tmem_st32(t_s, w);
        tmem_st32(t_s + 32, w + 32);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_bar.p_full[i]);
      }
      float l0, l1;
      upk2(l2, l0, l1);
      const float l = __fadd_rn(l0, l1), inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
      if (nb > 0) {
        wait(&s_bar.o_full[i], used++, abort);
        tc_fence_after();
      }
      if (lo > 0 || nb < all) {                  // to be joined with other blocks' sums
        Part *const part = parts + 2 * blockIdx.x + (lo == 0 ? 1 : 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[32];
          tmem_ask32(t_o + 32 * k, o);
          tmem_wait32(o);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            part->sums[i][8 * k + e][row] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                        __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
        }
        part->stat[i][row] = make_float2(m, l);
      } else {
        // through shared memory, so that a store of the warp covers whole lines: 16-byte pieces of 64
        // dimensions a row, the pieces of 8 rows permuted against one another
        const int64_t at0 = at - (int64_t)lane * a.Hq;           // the warp's first row
        const int live = n - (row - lane);                       // its rows
        uint4 *const out = static_cast<uint4 *>(a.out);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t o[2][32];
#pragma unroll
          for (int k = 0; k < 2; ++k) tmem_ask32(t_o + 64 * half + 32 * k, o[k]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            tmem_wait32(o[k]);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int f = 0; f < 4; ++f)
                w[f] = nb == 0 ? 0u : round_pair<KIND>(__fmul_rn(__uint_as_float(o[k][e + 2 * f]), inv),
                                                       __fmul_rn(__uint_as_float(o[k][e + 2 * f + 1]), inv));
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               staged + lane * 128 + (((4 * k + e / 8) ^ (lane & 7)) * 16)),
                           "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          __syncwarp();
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const int r = 4 * t + (lane >> 3);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(staged + r * 128 + (((lane & 7) ^ (r & 7)) * 16))
                         : "memory");
            if (r < live) out[(at0 + (int64_t)r * a.Hq) * (kTile / 8) + 8 * half + (lane & 7)] = v;
          }
          __syncwarp();
        }
        if (row < n && a.lse != nullptr) a.lse[at] = lse_of(m, l, c);
      }
      if (nb > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_bar.o_empty[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_abort) atomicOr(a.status, (uint32_t)HQ_ERR_TIMEOUT);
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The rows of tiles that several pieces share: a block a (piece that such a tile begins in, tile,
// 32 dimensions), a thread a row; the pieces' sums in order.
template <int KIND, bool CAP>
__global__ void __launch_bounds__(kPromptRows)
    prompt_join_kernel(PromptArgs a, const Plan *plan, const Item *list, const Part *parts) {
  follow_launch();
  const int first = blockIdx.x, i = blockIdx.y, k = blockIdx.z, row = threadIdx.x;
  if (plan->per == 0) return;
  const int4 job = plan->join[first];
  if (job.w == 0) return;
  const Item x = list[job.x];
  const int n = i == 0 ? x.n[0] : x.n[1], nb = blocks_of(i == 0 ? x.seen[0] : x.seen[1], n);
  if (nb <= job.z || row >= n) return;           // whole in the first piece
  const int more = min(job.w, (nb - job.z + plan->per - 1) / plan->per);
  const float c = factor_of<CAP>(a);
  const auto part = [&](int p) { return parts + 2 * (first + p) + (p == 0 ? 1 : 0); };
  float m = -INFINITY;
  for (int p = 0; p <= more; ++p) m = fmaxf(m, part(p)->stat[i][row].x);
  float l = 0.0f;
  float4 sum[8] = {};
#pragma unroll 2
  for (int p = 0; p <= more; ++p) {
    const float2 st = part(p)->stat[i][row];
    const float by = st.x == -INFINITY ? 0.0f : ex2(__fmul_rn(__fsub_rn(st.x, m), c));
    l = __fmaf_rn(st.y, by, l);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float4 v = part(p)->sums[i][8 * k + e][row];
      sum[e].x = __fmaf_rn(v.x, by, sum[e].x);
      sum[e].y = __fmaf_rn(v.y, by, sum[e].y);
      sum[e].z = __fmaf_rn(v.z, by, sum[e].z);
      sum[e].w = __fmaf_rn(v.w, by, sum[e].w);
    }
  }
  const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);
  const int h = job.y * a.G + (i == 0 ? x.head[0] : x.head[1]);
  const int64_t at = (int64_t)((i == 0 ? x.q[0] : x.q[1]) + row) * a.Hq + h;
  uint4 *const out = static_cast<uint4 *>(a.out) + at * (kTile / 8) + 4 * k;
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    out[e / 2] = make_uint4(round_pair<KIND>(__fmul_rn(sum[e].x, inv), __fmul_rn(sum[e].y, inv)),
                            round_pair<KIND>(__fmul_rn(sum[e].z, inv), __fmul_rn(sum[e].w, inv)),
                            round_pair<KIND>(__fmul_rn(sum[e + 1].x, inv), __fmul_rn(sum[e + 1].y, inv)),
                            round_pair<KIND>(__fmul_rn(sum[e + 1].z, inv), __fmul_rn(sum[e + 1].w, inv)));
  if (k == 0 && a.lse != nullptr) a.lse[at] = lse_of(m, l, c);
}

constexpr size_t kPlanBytes = (sizeof(Plan) + 255) / 256 * 256;
size_t list_bytes(int64_t room) { return ((size_t)room * sizeof(Item) + 255) / 256 * 256; }

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// Rows [tokens][heads][128] in boxes of 128 tokens of one head and 64 dimensions.
bool map_rows(CUtensorMap *map, const void *p, int kind, int64_t token, int64_t head, int tokens, int heads) {
  const cuuint64_t dims[3] = {(cuuint64_t)kTile, (cuuint64_t)heads, (cuuint64_t)tokens};
  // a stride that nothing goes by still has to be one
  const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? head : kTile) * 2, (cuuint64_t)(tokens > 1 ? token : kTile) * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)kPromptRows}, step[3] = {1, 1, 1};
  const EncodeTiled f = encode_tiled();
  return f != nullptr &&
         f(map, kind == HQ_T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(p),
           dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, bool CAP>
int launch(const PromptArgs &a, cudaStream_t st) {
  PromptMaps maps;
  if (!map_rows(&maps.q, a.q, a.kind, a.q_token, a.q_head, a.n_tokens, a.Hq)) return 1;
  if (a.n_k_tokens > 0) {
    if (!map_rows(&maps.k, a.k, a.kind, a.k_token, a.k_head, a.n_k_tokens, a.n_kv) ||
        !map_rows(&maps.v, a.v, a.kind, a.v_token, a.v_head, a.n_k_tokens, a.n_kv))
      return 1;
  } else {
    maps.k = maps.v = maps.q;                    // no item reads them
  }
  static int cache[64] = {};                     // multiprocessors, asked for once an instance and device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  int sms = dev < 64 ? cache[dev] : 0;
  if (sms == 0) {
    if (cudaFuncSetAttribute(prompt_kernel<KIND, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 1;
    }
    if (dev < 64) cache[dev] = sms;
  }
  const int64_t room = prompt_most_units(a.n_seqs, a.n_tokens, a.G);
  const bool split = may_split(room, a.n_kv, a.n_k_tokens);
  int grid = sms < kMostBlocks ? sms : kMostBlocks;
  if (!split && room * a.n_kv < grid) grid = (int)(room * a.n_kv);
  char *ws = static_cast<char *>(a.ws);
  Plan *plan = reinterpret_cast<Plan *>(ws);
  Item *list = reinterpret_cast<Item *>(ws + kPlanBytes);
  Part *parts = reinterpret_cast<Part *>(ws + kPlanBytes + list_bytes(room));
  const bool listed = split || room * a.n_kv > grid;
  if (listed &&
      launch_behind(prompt_prep_kernel, dim3(1), kPrepThreads, 0, st, a, plan, list, (int)room, grid, split ? 1 : 0) != 0)
    return 1;
  if (launch_behind(prompt_kernel<KIND, CAP>, dim3((unsigned)grid), kThreads, (size_t)kSmem, st, maps, a,
                    (const Plan *)(listed ? plan : nullptr), (const Item *)list, parts) != 0)
    return 1;
  if (!split) return 0;
  return launch_behind(prompt_join_kernel<KIND, CAP>, dim3((unsigned)grid, 2, 4), kPromptRows, 0, st, a, (const Plan *)plan,
                       (const Item *)list, (const Part *)parts);
}

}  // namespace

size_t prompt_workspace_bytes(int n_seqs, int64_t n_tokens, int Hq, int n_kv) {
  const int64_t room = prompt_most_units(n_seqs, n_tokens, Hq / n_kv);
  return kPlanBytes + list_bytes(room) + (may_split(room, n_kv, 16 * kKeys + 1) ? 2 * kMostBlocks * sizeof(Part) : 0);
}

int launch_prompt_attention(const PromptArgs &a, cudaStream_t st) {
  if (a.kind == HQ_T_BF16) return a.cap > 0.0f ? launch<HQ_T_BF16, true>(a, st) : launch<HQ_T_BF16, false>(a, st);
  return a.cap > 0.0f ? launch<HQ_T_F16, true>(a, st) : launch<HQ_T_F16, false>(a, st);
}

}  // namespace hq
