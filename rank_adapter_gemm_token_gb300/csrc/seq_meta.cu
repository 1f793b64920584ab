// One step's sequences: the metadata that every layer's cache write, attention and cache read of the
// step share (mlora_build_seq). Two launches:
//   check   a warp for each sequence: its bounds (inside the step, not below an earlier start) and its
//           page table (every page of its cached length inside the cache), the used part of the table
//           copied into the step's own storage, so that the caller's may change as soon as this kernel
//           has run. A sequence that fails is skipped
//           (length 0: nothing is read or written for it, its rows of the attention are zero) and
//           recorded;
//   plan    blocks 0 and 1: the work of the row kernel and of the tile kernel as prefix sums, over which their CTAs take
//           equal shares, or whole items dealt out, where there are enough (tile kernel, whose CTAs get lists); the other
//           blocks: sequence, position and cache row of each token.
// Bound by latency: a few dependent loads, block scans and searches; the table is read once. Measured on the GPU: 7.4 us for 256
// single tokens, 9.8 with four chunks beside them, 25 for 300 prompts of 100 tokens (4800 items), once for all layers of a step.
#include <algorithm>
#include <climits>
#include <cstddef>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kCheckThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kMaxLen = INT_MAX - 255;   // so that a length rounded up to whole pages, units or tiles is an int
constexpr int kMapSeqs = 8192;      // MLORA_MAX_SEQS: token starts kept in shared memory by the token map
constexpr int kPlanPre = kMapSeqs / 2;   // prefix sums kept there by the plan

__global__ void __launch_bounds__(kCheckThreads)
check_seq_kernel(const int32_t* __restrict__ q_start, const int32_t* __restrict__ kv_len,
                 const int32_t* __restrict__ pages, int table_ld, SeqView v, int max_new, int n_pages, int page_log2) {
  constexpr int kSeqs = kCheckThreads / 32;
  __shared__ int32_t tops[kSeqs];
  ptx::grid_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s0 = blockIdx.x * kSeqs, s = s0 + warp;
  // The largest start up to the sequence's own: one below an earlier start would share tokens with another sequence, and
  // accepted sequences could have more than T tokens in all, which is what the plan's lists hold.
  int top = INT_MIN;
  for (int i = threadIdx.x; i < s0; i += kCheckThreads) top = max(top, q_start[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
  if (s >= v.S) return;
  top = __reduce_max_sync(0xffffffffu, lane < kSeqs ? max(tops[lane], lane <= warp ? q_start[s0 + lane] : INT_MIN) : INT_MIN);
  const int a = q_start[s], b = q_start[s + 1], L = kv_len[s];
  const int page = 1 << page_log2;
  bool ok = a >= 0 && a == top && a <= b && b <= v.T && b - a <= max_new && L >= 0 && L <= kMaxLen &&
            static_cast<int64_t>(L) <= static_cast<int64_t>(v.max_pages) * page && (L == 0 || L >= b - a);
  const int used = ok ? (L + page - 1) >> page_log2 : 0;
  bool fine = true;
  for (int i = lane; i < used; i += 32) {
    const int p = pages[static_cast<size_t>(s) * table_ld + i];
    fine = fine && p >= 0 && p < n_pages;
    v.table[static_cast<size_t>(s) * v.max_pages + i] = p;
  }
  ok = __all_sync(0xffffffffu, fine) && ok;
  if (lane == 0) {
    v.start[s] = ok ? a : 0;
    v.n[s] = ok ? b - a : 0;
    v.len[s] = ok ? L : 0;
    if (!ok) {
      atomicOr(v.err, ptx::kErrBadSeq);
      atomicMin(&v.counts[1], s);
    }
  }
}

// Inclusive scans of N values over the block's kPlanThreads threads, in place; total gets the sums.
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&x)[N], int64_t (*warp_sums)[32], int64_t (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[i], d);
      if (lane >= d) x[i] += y;
    }
    if (lane == 31) warp_sums[i][warp] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int64_t w = warp_sums[i][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    total[i] = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    if (warp > 0) x[i] += before;
  }
  __syncthreads();
}

// x[i] <- max(x[0], ..., x[i]), i < n, by all threads of the block, a run of elements each; tops: a place for each thread.
__device__ __noinline__ void running_max(int32_t* x, int n, int32_t* tops) {
  const int per = (n + kPlanThreads - 1) / kPlanThreads, i0 = min(static_cast<int>(threadIdx.x) * per, n), i1 = min(i0 + per, n);
  int32_t top = INT_MIN;
  for (int i = i0; i < i1; ++i) x[i] = top = max(top, x[i]);
  tops[threadIdx.x] = top;
  for (int d = 1; d < kPlanThreads; d <<= 1) {
    __syncthreads();
    const int32_t before = static_cast<int>(threadIdx.x) >= d ? tops[threadIdx.x - d] : INT_MIN;
    __syncthreads();
    tops[threadIdx.x] = max(tops[threadIdx.x], before);
  }
  __syncthreads();
  if (threadIdx.x > 0)
    for (int i = i0; i < i1; ++i) x[i] = max(x[i], tops[threadIdx.x - 1]);
  __syncthreads();
}

// The last i in [0, n) with pre[i] <= x, by one thread.
__device__ int last_below(const int64_t* pre, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// One cut of a list of `n` entries with prefix sums pre: where it falls (entry, head, unit of the item), and the item
// if the cut is the first inside it.
struct Cut {
  int item, kvh, unit;
  int64_t at;
  JoinTask join;
};
__device__ Cut cut_at(const Shares& sh, const int64_t* pre, int n, int Hkv, int64_t c) {
  Cut r{n, 0, 0, sh.total, JoinTask{0, 0, 0, 0}};
  const int64_t y = sh.raw(c);
  if (y >= sh.total) return r;
  r.item = last_below(pre, n, y);
  const int units = static_cast<int>((pre[r.item + 1] - pre[r.item]) / Hkv);
  r.kvh = static_cast<int>(y - pre[r.item]) / units;
  const int64_t a = pre[r.item] + static_cast<int64_t>(r.kvh) * units, b = a + units;
  r.at = sh.snapped(y, a, b);
  if (r.at > a && r.at < b) {
    int first, cuts;
    sh.inside(a, b, &first, &cuts);
    r.join = JoinTask{r.item, r.kvh, first, cuts + 1};
    r.unit = static_cast<int>(r.at - a);
  } else if (r.at == b) {              // the next item
    if (++r.kvh == Hkv) r.kvh = 0, ++r.item;
  }
  return r;
}

// Key tiles [ka, kb) of an item, to a place of a list.
__device__ __forceinline__ void put_work(const SeqView& v, int64_t place, const TileBlk& b, int kvh, int ka, int kb) {
  int end[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int from = b.t0 + v.tile_tokens * w, last = min(from + v.tile_tokens, b.n) - 1;
    end[w] = from < b.n ? max(ka, min(kb, (b.len - b.n + last) / kTileKeys + 1)) : ka;
  }
  int4* to = reinterpret_cast<int4*>(v.tile_work + place);
  to[0] = make_int4(ka, kb, end[0], end[1]);
  to[1] = make_int4(b.len, b.n, b.start, b.t0);
  to[2] = make_int4(b.seq, kvh, ka > 0 || kb < b.tiles, 0);
}
static_assert(sizeof(TileWork) == 48 && offsetof(TileWork, len) == 16 && offsetof(TileWork, seq) == 32, "written in this order");

// The shares and joins of one list of n entries; cuts, parts: places for kPlanThreads cuts' positions and items' parts.
template <bool TILES>
__device__ __forceinline__ void share_out(const SeqView& v, const int64_t* pre, int n, const Shares& sh, int ctas, int64_t* cuts,
                                          int64_t* parts, int* joins) {
  const int c = threadIdx.x;
  Cut cut{n, 0, 0, sh.total, JoinTask{0, 0, 0, 0}};
  if (c <= sh.n && sh.total > 0) cut = cut_at(sh, pre, n, v.Hkv, c);
  // A row CTA counts units of keys alone: those of an item's head are taken off where the item begins. A tile CTA gets a
  // list: the cut as the item's number and the key tile in it.
  const int64_t number = static_cast<int64_t>(cut.item) * v.Hkv + cut.kvh;
  cuts[c] = TILES ? number << 32 | max(cut.unit - kTileHead, 0) : cut.at - kRowHead * (number + (cut.unit > 0));
  __syncthreads();
  if (!TILES) {                                   // (the prefix sums are not wanted any more)
    parts[c] = static_cast<int64_t>(cut.join.cta) << 32 | cut.join.parts;
    __syncthreads();
  }
  if (!TILES && c < ctas) {
    const int units = c < sh.n && sh.total > 0 ? static_cast<int>(cuts[c + 1] - cuts[c]) : 0;
    const int64_t next = parts[c + 1];
    v.row_share[c] = RowShare{cut.item, cut.kvh, max(cut.unit - kRowHead, 0), units, cut.join.cta, cut.join.parts,
                              static_cast<int>(next >> 32), static_cast<int>(next)};
    v.row_there[c] = v.row_there[ctas + c] = v.row_there[2 * ctas + c] = 0;
  }
  if (TILES) {
    // a warp to a CTA's list; before it lie that many items and one place for each cut
    for (int k = threadIdx.x >> 5; k < ctas; k += kPlanThreads / 32) {
      const bool some = k < sh.n && sh.total > 0;
      const int64_t from = cuts[k], to = some ? cuts[k + 1] : from;
      const int first = static_cast<int>(from >> 32), ka = static_cast<int>(from), kb = static_cast<int>(to);
      const int count = static_cast<int>(to >> 32) - first + (kb > 0);
      const int place = first + k;
      for (int i = threadIdx.x & 31; i < count; i += 32) {
        const TileBlk b = v.blk[(first + i) / v.Hkv];
        put_work(v, place + i, b, (first + i) % v.Hkv, i == 0 ? ka : 0, i == count - 1 && kb > 0 ? kb : b.tiles);
      }
      if ((threadIdx.x & 31) == 0) v.tile_share[k] = make_int2(place, some ? count : 0);
    }
  }
  if (TILES && cut.join.parts > 0 && c == cut.join.cta + 1) v.tile_join[atomicAdd(joins, 1)] = cut.join;
  __syncthreads();
}

// The row kernel's work, or the tile kernel's (TILES).
template <bool TILES>
__device__ void plan(const SeqView& v, int page_log2, int64_t* pre, int64_t* cuts) {
  __shared__ int64_t sums[4][32];
  __shared__ int joins;                           // split items so far (their order in the lists does not matter)
  __shared__ int most, deepest;                   // key tiles of the largest block; units of the fullest hands
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t units = 0, entries = 0, cached = 0, blocks = 0;      // totals of the sequences before this chunk
  for (int s0 = 0; s0 < v.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const int n = s < v.S ? v.n[s] : 0, L = s < v.S ? v.len[s] : 0, start = s < v.S ? v.start[s] : 0;
    const int64_t rows = static_cast<int64_t>(n) * v.G;
    const bool some = rows > 0 && L > 0, few = rows <= v.row_limit;
    const int per = 2 * v.tile_tokens;              // tokens of a block
    const int64_t u = some && few ? kRowHead + (L + kRowUnit - 1) / kRowUnit : 0;
    const int64_t b = some && !few ? (n + per - 1) / per : 0;
    int64_t x[4] = {u, u > 0, (static_cast<int64_t>(L) + (1 << page_log2) - 1) >> page_log2, b}, t[4];
    block_scan(x, sums, t);
    if (!TILES && s < v.S) v.page_pre[s + 1] = static_cast<int32_t>(cached + x[2]);
    if (!TILES && u > 0) {
      const int64_t e = entries + x[1];
      v.row_seq[e - 1] = RowSeq{s, n, L, start};
      v.row_pre[e] = (units + x[0]) * v.Hkv;
    }
    // the chunk's tile blocks, a warp for each sequence
    const int64_t first = blocks + x[3] - b;
    uint32_t has = __ballot_sync(0xffffffffu, TILES && b > 0);
    while (has) {
      const int i = __ffs(has) - 1;
      has &= has - 1;
      const int nb = static_cast<int>(__shfl_sync(0xffffffffu, b, i)), bn = __shfl_sync(0xffffffffu, n, i),
                bl = __shfl_sync(0xffffffffu, L, i), bstart = __shfl_sync(0xffffffffu, start, i);
      const int64_t f = __shfl_sync(0xffffffffu, first, i);
      for (int k = lane; k < nb; k += 32) {
        const int tiles = (bl - bn + min((k + 1) * per, bn) - 1) / kTileKeys + 1;
        v.blk[f + k] = TileBlk{s0 + warp * 32 + i, bn, bl, bstart, k * per, tiles};
      }
    }
    units += t[0];
    entries += t[1];
    cached += t[2];
    blocks += t[3];
  }
  if (threadIdx.x == 0) {
    if (!TILES) v.row_pre[0] = v.page_pre[0] = 0;
    if (TILES) v.blk_pre[0] = 0;
    joins = most = deepest = 0;
  }
  __syncthreads();
  // The prefix sums once more in shared memory, where they fit: the cuts are searched in them.
  if (!TILES) {
    const bool small_rows = entries < kPlanPre;
    if (small_rows)
      for (int64_t i = threadIdx.x; i <= entries; i += kPlanThreads) pre[i] = v.row_pre[i];
    __syncthreads();
    const int64_t row_total = units * v.Hkv;
    share_out<false>(v, small_rows ? pre : v.row_pre, static_cast<int>(entries),
                     Shares{row_total, static_cast<int>(min(static_cast<int64_t>(v.row_ctas), row_total)), kRowHead, 0}, v.row_ctas,
                     cuts, pre, &joins);
    return;
  }
  int64_t tiles = 0;
  const bool small_tiles = blocks < kPlanPre;
  for (int64_t j0 = 0; j0 < blocks; j0 += kPlanThreads) {
    const int64_t j = j0 + threadIdx.x;
    const int size = j < blocks ? v.blk[j].tiles : 0, high = __reduce_max_sync(0xffffffffu, size);
    if (lane == 0) atomicMax(&most, high);
    int64_t x[1] = {j < blocks ? kTileHead + size : 0}, t[1];
    block_scan(x, sums, t);
    if (j < blocks) {
      const int64_t p = (tiles + x[0]) * v.Hkv;
      v.blk_pre[j + 1] = p;
      if (small_tiles) pre[j + 1] = p;
    }
    tiles += t[0];
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  const int64_t tile_total = tiles * v.Hkv, items = blocks * v.Hkv;
  // Whole items dealt out by falling size, the hands going to the CTAs forwards and backwards in turn, come within the first
  // item of the last hand of equal work, without parts to join; where they would be further off (few items, or large ones
  // among the last), equal shares split and join. Whole items against shares, bf16: 8 x 512 tokens 36 us against 42, one
  // prompt of 8000 335 against 364, 6 chunks of 300 tokens on 4000 108 against 132 (there the fullest hands lie 12 units
  // above the mean: the shares' own distance, since an item's cost follows its units only roughly).
  const int n = v.tile_ctas;
  if (items >= n && items < (1 << 28)) {
    const int shift = max(0, 22 - __clz(most));     // sizes in 1024 classes
    int* at = reinterpret_cast<int*>(cuts);         // blocks of each class, the larger first; then where they go
    at[threadIdx.x] = 0;
    __syncthreads();
    // The blocks' next places in their classes; a warp's blocks of one class (often all of them) take theirs together.
    auto places = [&](int64_t* rank) {
      for (int64_t j0 = 0; j0 < blocks; j0 += kPlanThreads) {
        const int64_t j = j0 + threadIdx.x;
        const int cls = j < blocks ? 1023 - (v.blk[j].tiles >> shift) : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, cls);
        const int leader = __ffs(same) - 1;
        int first = 0;
        if (lane == leader && cls >= 0) first = atomicAdd(&at[cls], __popc(same));
        first = __shfl_sync(0xffffffffu, first, leader);
        if (rank != nullptr && cls >= 0) rank[j] = first + __popc(same & ((1u << lane) - 1));
      }
    };
    places(nullptr);
    __syncthreads();
    const int own = at[threadIdx.x], hands = static_cast<int>((items + n - 1) / n);
    int64_t x[1] = {own}, t[1];
    block_scan(x, sums, t);
    at[threadIdx.x] = static_cast<int>(x[0]) - own;
    __syncthreads();
    auto size = [&](int i) {                        // units of the i-th item by falling size
      const int rank = i / v.Hkv;
      int lo = 0, hi = 1024;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= rank) lo = mid; else hi = mid;
      }
      return kTileHead + ((1024 - lo) << shift) - 1;
    };
    const int64_t mean = tile_total / n;
    if (threadIdx.x < n) {
      int64_t sum = 0;
      if (hands <= 8) {
        for (int h = 0; h < hands; ++h) {
          const int i = h * n + static_cast<int>((h & 1) != 0 ? n - 1 - threadIdx.x : threadIdx.x);
          if (i < items) sum += size(i);
        }
      } else if (threadIdx.x == 0) {
        sum = max(static_cast<int64_t>(size(0)), mean + size((hands - 1) * n));
      }
      atomicMax(&deepest, static_cast<int>(min(sum, static_cast<int64_t>(INT_MAX))));
    }
    __syncthreads();
    if (deepest <= mean + kTileDeal) {
      // (which block of a class comes first changes who does an item, not how it is done)
      int64_t* rank = small_tiles ? pre : v.blk_pre;           // (its prefix sums are not wanted)
      places(rank);
      __syncthreads();
      for (int i = threadIdx.x; i < static_cast<int>(items); i += kPlanThreads) {
        const int j = i / v.Hkv, kvh = i - j * v.Hkv, place = static_cast<int>(rank[j]) * v.Hkv + kvh;
        const int hand = place / n, c = place - hand * n, cta = (hand & 1) != 0 ? n - 1 - c : c;
        const TileBlk b = v.blk[j];
        put_work(v, cta * hands + hand, b, kvh, 0, b.tiles);
      }
      const int over = static_cast<int>(items - static_cast<int64_t>(hands - 1) * n);      // items of the last hand
      for (int cta = threadIdx.x; cta < n; cta += kPlanThreads) {
        const int c = ((hands - 1) & 1) != 0 ? n - 1 - cta : cta;
        v.tile_share[cta] = make_int2(cta * hands, hands - (c < over ? 0 : 1));
      }
      if (threadIdx.x == 0) v.counts[2] = 0;
      return;
    }
  }
  share_out<true>(v, small_tiles ? pre : v.blk_pre, static_cast<int>(blocks),
                  Shares{tile_total, static_cast<int>(min(static_cast<int64_t>(v.tile_ctas), tile_total)), kTileHead, kTileSnap},
                  v.tile_ctas, cuts, pre, &joins);
  if (threadIdx.x == 0) v.counts[2] = joins;
}

__global__ void __launch_bounds__(kPlanThreads)
plan_seq_kernel(const int32_t* __restrict__ q_start, SeqView v, int page_log2) {
  __shared__ alignas(16) int32_t begin[kMapSeqs + 1];
  __shared__ int64_t cuts[kPlanThreads];
  const int S = v.S;
  bool falls = false;
  if (blockIdx.x > 1)
    for (int i = threadIdx.x; i <= S && S > 0; i += kPlanThreads) {
      begin[i] = q_start[i];
      falls = falls || (i > 0 && q_start[i - 1] > begin[i]);
    }
  ptx::grid_dependency_wait();        // the check's results
  if (blockIdx.x < 2) {
    int64_t* pre = reinterpret_cast<int64_t*>(begin);
    if (blockIdx.x == 0)
      plan<false>(v, page_log2, pre, cuts);
    else
      plan<true>(v, page_log2, pre, cuts);
    return;
  }
  // Starts that fall somewhere: their running maximum takes their place, which is an accepted sequence's own start and its end.
  if (__syncthreads_or(falls)) running_max(begin, S + 1, reinterpret_cast<int32_t*>(cuts));
  const int t = (blockIdx.x - 2) * kPlanThreads + threadIdx.x;
  if (t >= v.T) return;
  int lo = 0, hi = S;                 // the last s with begin[s] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (begin[mid] <= t) lo = mid; else hi = mid;
  }
  int seq = -1, pos = 0, row = -1;
  if (S > 0 && begin[lo] <= t && t < begin[lo + 1]) {
    const int L = v.len[lo];
    if (L > 0) {
      seq = lo;
      pos = L - v.n[lo] + (t - begin[lo]);
      const int p = v.table[static_cast<size_t>(lo) * v.max_pages + (pos >> page_log2)];
      row = (p << page_log2) + (pos & ((1 << page_log2) - 1));
    }
  }
  v.tok_seq[t] = seq;
  v.tok_pos[t] = pos;
  v.tok_row[t] = row;
}

}  // namespace

cudaError_t launch_build_seq(const int32_t* q_start, const int32_t* kv_len, const int32_t* pages, int table_ld,
                             const SeqView& s, int max_new, const KvView& kv, cudaStream_t st) {
  const int check = std::max(1, (s.S + kCheckThreads / 32 - 1) / (kCheckThreads / 32));
  note_launch_begin(kKindSeq, st);
  check_seq_kernel<<<check, kCheckThreads, 0, st>>>(q_start, kv_len, pages, table_ld, s, max_new, kv.n_pages,
                                                    kv.page_log2);
  cudaError_t e = cudaGetLastError();
  note_launch_end(kKindSeq, st);
  if (e != cudaSuccess) return e;
  note_launch_begin(kKindSeq, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 + (s.T + kPlanThreads - 1) / kPlanThreads);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, plan_seq_kernel, q_start, s, kv.page_log2);
  note_launch_end(kKindSeq, st);
  return e;
}

}  // namespace mlora
