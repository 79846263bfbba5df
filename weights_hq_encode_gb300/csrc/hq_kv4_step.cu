// hq_kv4_step.cu -- what a serving step does to the 4-bit window cache's
// bookkeeping (include/hq_kv4.h): pages and slots for sequences that grow or
// shrink, and the accepted path of a tree of drafted tokens.
#include <atomic>

#include <cuda_runtime.h>

#include "hq_kv4.h"
#include "hq_launch.cuh"

namespace hq {

namespace {

// ------------------------------------------------------------------ resize
// Exclusive sums of two values a thread over the block, and their totals.
template <int THREADS>
__device__ void block_scan2(int64_t &x, int64_t &y, int64_t &all_x, int64_t &all_y, int64_t (*s_warp)[2]) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t ox = __shfl_up_sync(0xffffffffu, x, d), oy = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += ox;
      y += oy;
    }
  }
  if (lane == 31) {
    s_warp[warp][0] = x;
    s_warp[warp][1] = y;
  }
  __syncthreads();
  int64_t wx = lane < kWarps ? s_warp[lane][0] : 0, wy = lane < kWarps ? s_warp[lane][1] : 0;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const int64_t ox = __shfl_up_sync(0xffffffffu, wx, d), oy = __shfl_up_sync(0xffffffffu, wy, d);
    if (lane >= d) {
      wx += ox;
      wy += oy;
    }
  }
  all_x = __shfl_sync(0xffffffffu, wx, kWarps - 1);
  all_y = __shfl_sync(0xffffffffu, wy, kWarps - 1);
  const int64_t bx = __shfl_sync(0xffffffffu, wx, (warp + 31) & 31), by = __shfl_sync(0xffffffffu, wy, (warp + 31) & 31);
  x += (warp == 0 ? 0 : bx) - x0;
  y += (warp == 0 ? 0 : by) - y0;
}

// The sequence that holds rank r: the first whose end is behind it.
__device__ __forceinline__ int rank_owner(const int *ends, int n, int64_t r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

struct Change {
  int old, wanted;                               // lengths
  int have, want;                                // pages
  bool bad;
};
__device__ __forceinline__ Change change_of(const Kv4ResizeArgs &a, int b) {
  Change c;
  const int64_t cap = (int64_t)a.width * a.page_tokens;
  const int o = a.lengths[b], w = a.wanted[b];
  c.old = o < 0 ? 0 : o > cap ? (int)cap : o;
  c.wanted = w < 0 ? 0 : w > cap ? (int)cap : w;
  c.bad = c.old != o || c.wanted != w;
  c.have = (int)kv4_divide((int64_t)c.old + a.page_tokens - 1, a.page_tokens, a.page_shift);
  c.want = (int)kv4_divide((int64_t)c.wanted + a.page_tokens - 1, a.page_tokens, a.page_shift);
  return c;
}

// Every block adds up the whole batch (lengths come from L2) and writes its
// share of the lists and pages, so that blocks need nothing of one another: ranks
// among the pages given back, the pages taken and the new tokens are prefix
// sums over the sequences, and a rank's sequence is found by bisection in
// shared memory.  The i-th page taken is the i-th given back while there are
// such, then the i-th from the list's end: no block reads a place of the list
// or table that another writes, but for the list's length.  With several blocks that, the
// new lengths and the starts are a second launch's (`sums`), which adds up beside the
// first and writes when it has ended.
// Bound by latency: one load of the lengths, two scans, one search; 64 sequences and 517
// tokens 4 us, 512 sequences and 770 000 tokens 12 us (two launches).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv4_resize_kernel(Kv4ResizeArgs a) {
  extern __shared__ int s_ends[];                // [3][n_seqs]: given, taken, tokens
  __shared__ int64_t s_warp[2][THREADS / 32][2];
  // Either launch of two begins when all before both has ended: the first lets the second begin only then,
  // and the second, which reads what was there before the first, waits for that one before it writes.
  if (a.lists) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  const int n = a.n_seqs, tid = threadIdx.x;
  int *const s_give = s_ends, *const s_take = s_ends + n, *const s_tok = s_ends + 2 * n;
  const int per = (n + THREADS - 1) / THREADS;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  const bool first = blockIdx.x == 0;
  uint32_t bad = 0;
  int64_t n_free = *a.n_free;
  if (n_free < 0 || n_free > a.n_pages) {
    bad = HQ_ERR_PAGE;
    n_free = n_free < 0 ? 0 : a.n_pages;
  }
  int64_t at = 0, asked = 0, total, need;
  for (int b = b0; b < b1; ++b) {
    const Change c = change_of(a, b);
    if (c.bad) bad |= HQ_ERR_PAGE;
    at += max(0, c.have - c.want);
    asked += max(0, c.want - c.have);
  }
  block_scan2<THREADS>(at, asked, total, need, s_warp[0]);
  const int64_t given = min(total, a.n_pages - n_free);    // more cannot be in use
  if (total > given) bad |= HQ_ERR_PAGE;
  const int64_t avail = n_free + given;
  int64_t take_at = 0, tok_at = 0, taken, tokens;
  {
    int64_t demand = asked;
    for (int b = b0; b < b1; ++b) {
      const Change c = change_of(a, b);
      at += max(0, c.have - c.want);
      s_give[b] = (int)min(at, given);
      const int more = max(0, c.want - c.have);
      demand += more;
      const bool refused = more > 0 && demand > avail;
      if (refused) bad |= HQ_ERR_CAPACITY;
      take_at += refused ? 0 : more;
      tok_at += refused ? 0 : max(0, c.wanted - c.old);
    }
  }
  block_scan2<THREADS>(take_at, tok_at, taken, tokens, s_warp[1]);
  if (!a.lists) follow_launch();
  if (a.max_tokens < tokens && a.seq != nullptr) bad |= HQ_ERR_CAPACITY;
  if (a.sums && first && tid == 0 && a.starts != nullptr) a.starts[0] = 0;
  {
    int64_t demand = asked;
    for (int b = b0; b < b1; ++b) {
      const Change c = change_of(a, b);
      const int more = max(0, c.want - c.have);
      demand += more;
      const bool refused = more > 0 && demand > avail;
      take_at += refused ? 0 : more;
      tok_at += refused ? 0 : max(0, c.wanted - c.old);
      s_take[b] = (int)take_at;                  // at most avail
      s_tok[b] = (int)min(tok_at, (int64_t)INT32_MAX);
      if (a.sums && first) {
        a.new_lengths[b] = refused ? c.old : c.wanted;
        if (a.starts != nullptr) a.starts[b + 1] = (int)min(tok_at, (int64_t)INT32_MAX);
      }
    }
  }
  if (first && bad != 0) atomicOr(a.status, bad);
  __syncthreads();
  if (a.lists) {
    const int64_t step = (int64_t)gridDim.x * THREADS, me = (int64_t)blockIdx.x * THREADS + tid;
    bool bad_page = false;
    // pages: the g-th given back, from the place of its sequence and its place there
    const auto given_page = [&](int64_t g) {
      const int b = rank_owner(s_give, n, g);
      return a.table[(int64_t)b * a.width + change_of(a, b).want + (g - (b == 0 ? 0 : s_give[b - 1]))];
    };
    for (int64_t i = me; i < taken; i += step) {
      const int page = i < given ? given_page(i) : a.free_pages[n_free - 1 - (i - given)];
      if (page < 0 || page >= a.n_pages) bad_page = true;
      const int b = rank_owner(s_take, n, i);
      a.table[(int64_t)b * a.width + change_of(a, b).have + (i - (b == 0 ? 0 : s_take[b - 1]))] = page;
    }
    for (int64_t g = taken + me; g < given; g += step) {
      const int page = given_page(g);
      if (page < 0 || page >= a.n_pages) bad_page = true;
      a.free_pages[n_free + given - 1 - g] = page;
    }
    if (bad_page) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    // the new tokens, four a thread
    const int64_t listed = min(tokens, a.max_tokens);
    for (int64_t r = 4 * me; r < a.max_tokens; r += 4 * step) {
      int4 q = make_int4(-1, -1, -1, -1), p = make_int4(0, 0, 0, 0);
      int *const qs = &q.x, *const ps = &p.x;
      if (r < listed) {
        int b = rank_owner(s_tok, n, r);
        int end = s_tok[b], shift = change_of(a, b).old - (b == 0 ? 0 : s_tok[b - 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (r + k >= listed) break;
          while (r + k >= end) {                 // sequences without new tokens are skipped
            const int before = end;
            end = s_tok[++b];
            if (r + k < end) shift = change_of(a, b).old - before;
          }
          qs[k] = b;
          ps[k] = (int)(r + k) + shift;
        }
      }
      if (a.vec && r + 4 <= a.max_tokens) {
        *reinterpret_cast<int4 *>(a.seq + r) = q;
        *reinterpret_cast<int4 *>(a.pos + r) = p;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r + k < a.max_tokens) {
            a.seq[r + k] = qs[k];
            a.pos[r + k] = ps[k];
          }
      }
    }
  }
  if (a.sums && first && tid == 0) *a.n_free = (int)(avail - taken);
}

// ------------------------------------------------------------------ accept
// A warp moves the rows of one (sequence, head): lanes 0 .. 15 the 64 bytes of a
// row's K codes, lanes 16 .. 31 V's, a word each, the first lane of either half its scale.
// A lane always moves the same word of a row, and a row's new place is never
// behind its old one, while paths ascend: so no word is overwritten before it is
// read, in the order of the path, and nothing is shared between lanes.  Bound by the latency of
// lengths, path, table and rows, one behind the other: 64 sessions x 8 heads, paths of up to 64: 7 us.
constexpr int kAcceptWarps = 4, kAcceptAhead = 8;

__global__ void __launch_bounds__(32 * kAcceptWarps) kv4_accept_kernel(Kv4AcceptArgs a) {
  follow_launch();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * kAcceptWarps + (threadIdx.x >> 5);
  if (h >= a.c.n_kv) return;
  bool bad;
  const int L = kv4_length(a.c, a.lengths, b, &bad);
  const int32_t *path = a.path + (int64_t)b * a.max_path;
  const int half = lane >> 4, word = lane & 15;
  // V: chunk word / 2 of a token pair, the token's 8 bytes of it, word % 2 of them
  const auto code_at = [&](uint32_t place) {
    const int t = place % kUnit;
    return kv4_unit(a.c, place) + (half == 0 ? t * 64 + word * 4
                                             : kUnitV + (t >> 1) * 128 + (word >> 1) * 16 + (t & 1) * 8 + (word & 1) * 4);
  };
  const auto scale_at = [&](uint32_t place) {
    return kv4_unit(a.c, place) + (half == 0 ? kUnitKs : kUnitVs) + 2 * (place % kUnit);
  };
  int count = 0, last = -1;
  bool more = true;
  while (more && count < a.max_path) {           // 32 entries of the path at a time, an entry a lane
    const int i = count + lane, j = i < a.max_path ? path[i] : -1;
    int before = __shfl_up_sync(0xffffffffu, j, 1);
    if (lane == 0) before = last;
    // the path ends at its first entry that is negative, or not behind the one before, or past the capacity
    const bool wrong = j >= 0 && (j <= before || (int64_t)L + j >= a.c.capacity());
    const uint32_t ends = __ballot_sync(0xffffffffu, j < 0 || wrong);
    const int n = ends == 0 ? 32 : __ffs(ends) - 1;
    if (lane == n && wrong) bad = true;
    uint32_t from = kNoPlace, to = kNoPlace;
    if (lane < n && j != i) {
      from = kv4_place(a.c, b, L + j, h);
      to = kv4_place(a.c, b, L + i, h);
      if (from == kNoPlace || to == kNoPlace) {
        bad = true;
        from = kNoPlace;
      }
    }
    for (int k0 = 0; k0 < n; k0 += kAcceptAhead) {
      uint32_t code[kAcceptAhead];
      uint16_t scale[kAcceptAhead];
#pragma unroll
      for (int k = 0; k < kAcceptAhead; ++k) {
        const uint32_t p = __shfl_sync(0xffffffffu, from, k0 + k);     // lanes past n name no place
        if (p == kNoPlace) continue;
        code[k] = *reinterpret_cast<const uint32_t *>(code_at(p));
        if (word == 0) scale[k] = *reinterpret_cast<const uint16_t *>(scale_at(p));
      }
#pragma unroll
      for (int k = 0; k < kAcceptAhead; ++k) {
        if (__shfl_sync(0xffffffffu, from, k0 + k) == kNoPlace) continue;
        const uint32_t p = __shfl_sync(0xffffffffu, to, k0 + k);
        *reinterpret_cast<uint32_t *>(code_at(p)) = code[k];
        if (word == 0) *reinterpret_cast<uint16_t *>(scale_at(p)) = scale[k];
      }
    }
    count += n;
    last = __shfl_sync(0xffffffffu, j, 31);
    more = ends == 0;
  }
  if (h == 0 && lane == 0) a.new_lengths[b] = L + count;
  if (bad) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
}

}  // namespace

namespace {

// Lets the larger kernel have the shared memory of the most sequences, once a device and the same
// whatever the batch: 48 KB, what is there without asking, are for its static part too.
bool room_for_resize() {
  static std::atomic<bool> done[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && done[dev].load()) return true;
  if (cudaFuncSetAttribute(kv4_resize_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           3 * HQ_KV4_MAX_RESIZE * (int)sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (dev < 64) done[dev].store(true);
  return true;
}

}  // namespace

int launch_kv4_resize(const Kv4ResizeArgs &a, cudaStream_t st) {
  const size_t smem = 3 * (size_t)a.n_seqs * sizeof(int);
  const int64_t entries = (int64_t)a.n_seqs * a.width, most = a.max_tokens / 4 > entries / 4 ? a.max_tokens / 4 : entries / 4;
  // by the entries of the lists, and of the table, of which any may change: a small block has short barriers
  if (a.n_seqs <= 512 && most <= 4096) return launch_behind(kv4_resize_kernel<256>, dim3(1), 256, smem, st, a);
  if (!room_for_resize()) return 1;
  Kv4ResizeArgs w = a;
  w.sums = 0;
  const int64_t want = most / 1024 + 1;
  if (launch_behind(kv4_resize_kernel<1024>, dim3((unsigned)(want < 152 ? want : 152)), 1024, smem, st, w) != 0) return 1;
  w.sums = 1;
  w.lists = 0;
  return launch_behind(kv4_resize_kernel<1024>, dim3(1), 1024, smem, st, w);
}

int launch_kv4_accept(const Kv4AcceptArgs &a, cudaStream_t st) {
  return launch_behind(kv4_accept_kernel,
                       dim3((unsigned)a.c.n_seqs, (unsigned)((a.c.n_kv + kAcceptWarps - 1) / kAcceptWarps)),
                       32 * kAcceptWarps, 0, st, a);
}

}  // namespace hq
