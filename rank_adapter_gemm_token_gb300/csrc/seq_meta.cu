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
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kCheckThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kMapSeqs = 8192;      // MLORA_MAX_SEQS: token starts kept in shared memory by the token map

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

// Inclusive scan over the block's kPlanThreads threads; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t w = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return x + (warp > 0 ? before : 0);
}

__device__ void plan(const SeqView& v, int page_log2) {
  __shared__ int64_t sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t tokens = 0, units = 0, cached = 0, blocks = 0;      // totals of the sequences before this chunk
  for (int s0 = 0; s0 < v.S; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    int n = s < v.S ? v.n[s] : 0;
    const int L = s < v.S ? v.len[s] : 0;
    // starts that do not ascend could name more tokens than there are: the lists hold T
    int64_t tn;
    const int64_t in = block_scan(n, sums, &tn);
    if (tokens + in > v.T) {
      n = 0;
      atomicOr(v.err, ptx::kErrBadSeq);
      atomicMin(&v.counts[1], s);
    }
    const int64_t rows = static_cast<int64_t>(n) * v.G;
    const bool some = rows > 0 && L > 0;
    const int64_t u = some && rows <= v.row_limit ? (L + kRowUnit - 1) / kRowUnit : 0;
    const int64_t p = (L + (1 << page_log2) - 1) >> page_log2;
    const int64_t b = some && rows > v.row_limit ? (rows + kBlockRows - 1) / kBlockRows : 0;
    int64_t tu, tp, tb;
    const int64_t iu = block_scan(u, sums, &tu), ip = block_scan(p, sums, &tp), ib = block_scan(b, sums, &tb);
    if (s < v.S) {
      v.row_pre[s + 1] = (units + iu) * v.Hkv;
      v.page_pre[s + 1] = static_cast<int32_t>(cached + ip);
    }
    // the chunk's tile blocks, a warp for each sequence
    const int64_t first = blocks + ib - b;
    for (int i = 0; i < 32; ++i) {
      const int nb = static_cast<int>(__shfl_sync(0xffffffffu, b, i));
      const int64_t f = __shfl_sync(0xffffffffu, first, i);
      for (int k = lane; k < nb; k += 32) {
        v.blk_seq[f + k] = s0 + warp * 32 + i;
        v.blk_row[f + k] = k * kBlockRows;
      }
    }
    tokens += tn;
    units += tu;
    cached += tp;
    blocks += tb;
  }
  if (threadIdx.x == 0) {
    v.row_pre[0] = 0;
    v.page_pre[0] = 0;
    v.blk_pre[0] = 0;
    v.counts[0] = static_cast<int32_t>(blocks);
  }
  __syncthreads();
  int64_t tiles = 0;
  for (int64_t j0 = 0; j0 < blocks; j0 += kPlanThreads) {
    const int64_t j = j0 + threadIdx.x;
    int64_t kt = 0;
    if (j < blocks) {
      const int s = v.blk_seq[j];
      const int n = v.n[s], L = v.len[s];
      const int64_t last = min(static_cast<int64_t>(v.blk_row[j]) + kBlockRows, static_cast<int64_t>(n) * v.G) - 1;
      kt = (L - n + last / v.G + 1 + kTileKeys - 1) / kTileKeys;
    }
    int64_t total;
    const int64_t inc = block_scan(kt, sums, &total);
    if (j < blocks) v.blk_pre[j + 1] = (tiles + inc) * v.Hkv;
    tiles += total;
  }
}

__global__ void __launch_bounds__(kPlanThreads)
plan_seq_kernel(const int32_t* __restrict__ q_start, SeqView v, int page_log2) {
  __shared__ int32_t begin[kMapSeqs + 1];
  const int S = v.S;
  if (blockIdx.x > 0)
    for (int i = threadIdx.x; i <= S && S > 0; i += kPlanThreads) begin[i] = q_start[i];
  ptx::grid_dependency_wait();        // the check's results
  if (blockIdx.x == 0) {
    plan(v, page_log2);
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
