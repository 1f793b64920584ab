// One step's sequences: the metadata that every layer's cache write, attention and cache read of the
// step share (mlora_build_seq). Two launches:
//   check   a warp for each sequence: its bounds and its page table (every page of its cached length
//           inside the cache), the used part of the table copied into the step's own storage, so that
//           the caller's may change as soon as this kernel has run. A sequence that fails is skipped
//           (length 0: nothing is read or written for it, its rows of the attention are zero) and
//           recorded;
//   plan    block 0: the work of the attention kernels as prefix sums, over which their CTAs take equal
//           shares (attention_rows.cu); the other blocks: sequence, position and cache row of each token.
// Bound by latency: a few dependent loads and three block scans; the table is read once.
#include <algorithm>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kCheckThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kMapSeqs = 8192;      // MLORA_MAX_SEQS: token starts kept in shared memory by the token map
constexpr int kPlanPre = kMapSeqs / 2;   // prefix sums kept there by the plan

__global__ void __launch_bounds__(kCheckThreads)
check_seq_kernel(const int32_t* __restrict__ q_start, const int32_t* __restrict__ kv_len,
                 const int32_t* __restrict__ pages, int table_ld, SeqView v, int max_new, int n_pages, int page_log2) {
  ptx::grid_dependents_launch();
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x * (kCheckThreads / 32) + (threadIdx.x >> 5);
  if (s >= v.S) return;
  const int a = q_start[s], b = q_start[s + 1], L = kv_len[s];
  const int page = 1 << page_log2;
  bool ok = a >= 0 && a <= b && b <= v.T && b - a <= max_new && L >= 0 &&
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
    if (c == first + 1) r.join = JoinTask{r.item, r.kvh, first, cuts + 1};
    r.unit = static_cast<int>(r.at - a);
  } else if (r.at == b) {              // the next item
    if (++r.kvh == Hkv) r.kvh = 0, ++r.item;
  }
  return r;
}

// The shares and joins of one list of n entries; cuts: a place for kPlanThreads + 1 cuts' positions.
template <bool TILES>
__device__ __forceinline__ void share_out(const SeqView& v, const int64_t* pre, int n, const Shares& sh, int ctas, int64_t* cuts,
                                          int* joins) {
  const int c = threadIdx.x;
  Cut cut{n, 0, 0, sh.total, JoinTask{0, 0, 0, 0}};
  if (c <= sh.n && sh.total > 0) cut = cut_at(sh, pre, n, v.Hkv, c);
  // (row shares count their keys' units alone: those of an item's head are taken off where the item begins)
  cuts[c] = TILES ? cut.at : cut.at - static_cast<int64_t>(kRowHead) * (static_cast<int64_t>(cut.item) * v.Hkv + cut.kvh + (cut.unit > 0));
  __syncthreads();
  if (c < ctas) {
    const int units = c < sh.n && sh.total > 0 ? static_cast<int>(cuts[c + 1] - cuts[c]) : 0;
    if (TILES)
      v.tile_share[c] = TileShare{cut.item, cut.kvh, max(cut.unit - kTileHead, 0), units};
    else
      v.row_share[c] = RowShare{cut.item, cut.kvh, max(cut.unit - kRowHead, 0), units};
  }
  if (cut.join.parts > 0) (TILES ? v.tile_join : v.row_join)[atomicAdd(joins, 1)] = cut.join;
  __syncthreads();
}

__device__ void plan(const SeqView& v, int page_log2, int64_t* pre) {
  __shared__ int64_t sums[5][32];
  __shared__ int64_t cuts[kPlanThreads];
  __shared__ int joins[2];                        // split items so far (their order in the lists does not matter)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t tokens = 0, units = 0, entries = 0, cached = 0, blocks = 0;      // totals of the sequences before this chunk
  for (int s0 = 0; s0 < v.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const int n = s < v.S ? v.n[s] : 0, L = s < v.S ? v.len[s] : 0, start = s < v.S ? v.start[s] : 0;
    const int64_t rows = static_cast<int64_t>(n) * v.G;
    const bool some = rows > 0 && L > 0, few = rows <= v.row_limit;
    const int per = 2 * v.tile_tokens;              // tokens of a block
    const int64_t u = some && few ? kRowHead + (L + kRowUnit - 1) / kRowUnit : 0;
    const int64_t b = some && !few ? (n + per - 1) / per : 0;
    int64_t x[5] = {n, u, u > 0, (static_cast<int64_t>(L) + (1 << page_log2) - 1) >> page_log2, b}, t[5];
    block_scan(x, sums, t);
    // starts that do not ascend could name more tokens than there are: the lists hold T
    const bool over = tokens + x[0] > v.T;
    if (over && n > 0) {
      atomicOr(v.err, ptx::kErrBadSeq);
      atomicMin(&v.counts[1], s);
    }
    if (s < v.S) v.page_pre[s + 1] = static_cast<int32_t>(cached + x[3]);
    if (u > 0) {
      const int64_t e = entries + x[2];
      v.row_seq[e - 1] = RowSeq{s, over ? 0 : n, L, start};
      v.row_pre[e] = (units + x[1]) * v.Hkv;
    }
    // the chunk's tile blocks, a warp for each sequence
    const int64_t first = blocks + x[4] - b;
    uint32_t has = __ballot_sync(0xffffffffu, b > 0);
    while (has) {
      const int i = __ffs(has) - 1;
      has &= has - 1;
      const int nb = static_cast<int>(__shfl_sync(0xffffffffu, b, i)), bn = __shfl_sync(0xffffffffu, n, i),
                bl = __shfl_sync(0xffffffffu, L, i), bstart = __shfl_sync(0xffffffffu, start, i);
      const int64_t f = __shfl_sync(0xffffffffu, first, i);
      if (__shfl_sync(0xffffffffu, static_cast<int>(over), i)) continue;
      for (int k = lane; k < nb; k += 32) {
        const int tiles = (bl - bn + min((k + 1) * per, bn) - 1) / kTileKeys + 1;
        v.blk[f + k] = TileBlk{s0 + warp * 32 + i, bn, bl, bstart, k * per, tiles};
      }
    }
    tokens += t[0];
    units += t[1];
    entries += t[2];
    cached += t[3];
    blocks += t[4];
    if (tokens > v.T) {                 // the rejected sequences' blocks are not there: the tile kernel leaves them all out
      blocks = 0;
      break;
    }
  }
  if (threadIdx.x == 0) {
    v.row_pre[0] = 0;
    v.page_pre[0] = 0;
    v.blk_pre[0] = 0;
    joins[0] = joins[1] = 0;
  }
  __syncthreads();
  // The prefix sums once more in shared memory, where they fit: the cuts are searched in them.
  const bool small_rows = entries < kPlanPre;
  if (small_rows)
    for (int64_t i = threadIdx.x; i <= entries; i += kPlanThreads) pre[i] = v.row_pre[i];
  __syncthreads();
  const int64_t row_total = units * v.Hkv;
  share_out<false>(v, small_rows ? pre : v.row_pre, static_cast<int>(entries),
                   Shares{row_total, static_cast<int>(min(static_cast<int64_t>(v.row_ctas), row_total)), kRowHead, 0}, v.row_ctas, cuts,
                   &joins[0]);
  int64_t tiles = 0;
  const bool small_tiles = blocks < kPlanPre;
  for (int64_t j0 = 0; j0 < blocks; j0 += kPlanThreads) {
    const int64_t j = j0 + threadIdx.x;
    int64_t x[1] = {j < blocks ? kTileHead + v.blk[j].tiles : 0}, t[1];
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
  const int64_t tile_total = tiles * v.Hkv;
  share_out<true>(v, small_tiles ? pre : v.blk_pre, static_cast<int>(blocks),
                  Shares{tile_total, static_cast<int>(min(static_cast<int64_t>(v.tile_ctas), tile_total)), kTileHead, kTileSnap},
                  v.tile_ctas, cuts, &joins[1]);
  if (threadIdx.x < 2) v.counts[2 + threadIdx.x] = joins[threadIdx.x];
}

__global__ void __launch_bounds__(kPlanThreads)
plan_seq_kernel(const int32_t* __restrict__ q_start, SeqView v, int page_log2) {
  __shared__ alignas(16) int32_t begin[kMapSeqs + 1];
  const int S = v.S;
  if (blockIdx.x > 0)
    for (int i = threadIdx.x; i <= S && S > 0; i += kPlanThreads) begin[i] = q_start[i];
  ptx::grid_dependency_wait();        // the check's results
  if (blockIdx.x == 0) {
    plan(v, page_log2, reinterpret_cast<int64_t*>(begin));
    return;
  }
  __syncthreads();
  const int t = (blockIdx.x - 1) * kPlanThreads + threadIdx.x;
  if (t >= v.T) return;
  int lo = 0, hi = S;                 // the last s with begin[s] <= t (the starts ascend, or are rejected below)
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
  cfg.gridDim = dim3(1 + (s.T + kPlanThreads - 1) / kPlanThreads);
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
