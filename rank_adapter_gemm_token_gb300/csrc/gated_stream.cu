// The gated linear of a few tokens (T <= 64): h = act(g) * u with [g u] = x W^T + the side path, in one launch that reads W once.
//
// Bound: HBM, the bytes of W (and of the adapters' rows in use): 2 to 128 flops a byte. So W goes from memory straight to registers,
// 16 bytes a lane and up to 8 steps ahead, and meets the tokens on the warp-level tensor instructions as their M side:
//   - a warp's 16 rows are 8 rows of the gate and the same 8 of the up projection, so that both values of an output lie in one
//     thread, which applies the activation. A quad's four lanes hold 32 consecutive k, eight each: the order of k inside a
//     product is free as long as both sides have the same, and so no operand is moved again. The tokens lie in shared memory
//     for the whole launch (rows 64 bytes off, so that a quarter warp's reads meet all banks).
//   - 12 warps stream, 8 columns of h each, dealt out to the SMs one after another; where that gives an SM fewer than 6 warps, 2
//     to 12 of them take a part of K each and add their sums up in shared memory, in order.
//   - the side path beside it, in the other 4 warps: v = A x for 16 rows of the adapters in use at a time. One or two such shares
//     (one token, rank 16) each CTA does for itself, without waiting for anyone; more are shared out among the CTAs by tickets
//     and handed around through the step's workspace (each CTA waits for all of them, a bounded wait: what has been drawn is
//     being worked on by a CTA that runs, and those that run draw until none is left). Then v is scaled and rounded to bf16,
//     as on the tensor-core side path. The columns of B of the slots in use follow the streaming warps' K loop as further k,
//     eight at a time, against v for the tokens that have the slot and 0 for the others.
// Measured on the GPU, 4096 -> 2 x 14336, L2 flushed before each call: one token, rank 16, 43 us, 5.4 TB/s (36 warm; pair GEMM 86);
// 16 tokens of 100 adapters 54 us (89); 20 tokens 62 (90). 64 tokens 1024 -> 2 x 14336 27 us (41). A token 1024 -> 2 x 2048 8.3 us
// (unfused, split-K kernel, 12.4). DRAM 69 % of its peak, issue slots 20 % (one token). Tried: v by the shrink kernel before it
// (16 tokens 59 us, its CTAs keep SMs from this one); 8 steps ahead with 18 warps (96 registers, spills: 50 us for one token).
#include <algorithm>

#include "attention.cuh"
#include "gated.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kWarps = 12;                  // that stream W
constexpr int kBuilders = 128;              // threads of the side path
constexpr int kStreamers = kWarps * 32, kThreads = kStreamers + kBuilders;
constexpr int kStep = 32;                   // k of a step: two products
constexpr int kWarpsWanted = 6;             // of an SM: 48 KB on their way, what the memory's latency asks for
template <int NT>
constexpr int kAhead = NT <= 2 ? 8 : NT <= 4 ? 6 : 4;     // steps on their way to a warp, 1 KB each, as far as the registers go
constexpr int kFetchPieces = 8;             // (of more, asking for them takes longer than it saves: 16 tokens 53.7 us, 58.4 with)
constexpr int kOwnShares = 2;               // shares of the side path up to which each CTA does all of them
// Named barriers: 1 ... kWarps / 2 of warps that share a group; of the three warps of the side path that look at the tokens' pairs, of
// the streaming warps, of both sides, of the side path
constexpr int kBarPairs = 12, kBarStream = 13, kBarTokens = 14, kBarSide = 15;

struct StreamPlan {
  int split;                                // warps that share a group of 8 columns
  int x_row;                                // bytes of a token's row
  int v_off, v_row, table_off, act, piece_off, pair_off, sum_off, part_off, bytes;
  int shares;                               // of the side path, at most
};

StreamPlan stream_plan(int T, int J, int K, int F, const PoolView& pool, int num_sms) {
  StreamPlan p{};
  p.split = kWarps;
  for (int s : {6, 4, 3, 2, 1})
    if (static_cast<int64_t>(F / 8) * s >= static_cast<int64_t>(kWarpsWanted) * num_sms) p.split = s;
  const int tiles = T <= 8 ? 1 : T <= 16 ? 2 : T <= 32 ? 4 : 8;
  const int64_t n = static_cast<int64_t>(T) * J;
  p.x_row = (K + 63) / 64 * 128 + 64;
  p.act = static_cast<int>(std::min<int64_t>(n, pool.S));
  p.v_row = pool.R * 2;
  p.shares = static_cast<int>((static_cast<int64_t>(p.act) * (pool.R / 8) + 1) / 2);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 15) / 16 * 16;
    return static_cast<int>(std::min<int64_t>(here, 1 << 30));
  };
  take(static_cast<int64_t>(T) * p.x_row);
  p.v_off = take(n * p.v_row);
  p.table_off = take(static_cast<int64_t>(T) * p.act * 2);
  p.piece_off = take(static_cast<int64_t>(p.act) * (pool.R / 8) * 8);
  p.pair_off = take(n * 8);
  p.sum_off = take(kBuilders * 4 * tiles * 4);
  p.part_off = take(p.split > 1 ? kStreamers * 4 * tiles * 4 : 0);
  p.bytes = static_cast<int>(std::min<int64_t>(at, 1 << 30));
  return p;
}

__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 k of 16 rows (the first eight in g, the others in u) against 8 tokens.
__device__ __forceinline__ void step(float (&d)[4], const uint4& g, const uint4& u, const uint4& x) {
  mma(d, g.x, u.x, g.y, u.y, x.x, x.y);
  mma(d, g.z, u.z, g.w, u.w, x.z, x.w);
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
gated_stream_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ W, uint16_t* __restrict__ h, int K, int F, int act,
                    PoolView pool, MetaView m, StreamPlan p, uint32_t* __restrict__ err) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int pieces, ticket;                      // groups of 8 columns of the slot space in use; the CTA's next share of them
  constexpr int N = kAhead<NT>;
  ptx::grid_dependents_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int T = m.T, steps = (K + kStep - 1) / kStep;
  int16_t* table = reinterpret_cast<int16_t*>(smem + p.table_off);        // [T][act] pair whose v a token has for an active slot (or -1)
  int2* piece = reinterpret_cast<int2*>(smem + p.piece_off);              // first column, active slot | eighth of the slot << 16
  const uint8_t* xrow[NT];                                                // (a column of no token repeats the last one)
#pragma unroll
  for (int z = 0; z < NT; ++z) xrow[z] = smem + static_cast<size_t>(min(8 * z + g, T - 1)) * p.x_row + t * 16;
  auto x_at = [&](int z, int s) { return *reinterpret_cast<const uint4*>(xrow[z] + s * kStep * 2); };
  float acc[NT][4];
  auto clear = [&]() {
#pragma unroll
    for (int z = 0; z < NT; ++z)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[z][i] = 0.f;
  };

  if (warp >= kWarps) {
    // ------------------------------------------------------------------ the side path
    const int tid = threadIdx.x - kStreamers, R = pool.R;
    float2* pairs = reinterpret_cast<float2*>(smem + p.pair_off);         // factor and rank (0: nothing) of each pair
    ptx::grid_dependency_wait();
    const bool alone = p.shares <= kOwnShares;
    const int n_act = min(m.counts[4], p.act);
    if (tid == 0) ticket = n_act > 0 && !alone ? static_cast<int>(atomicAdd(&m.sync[0], 1u)) : 0;
    if (warp == kWarps) {
      int before = 0;
      for (int a0 = 0; a0 < n_act; a0 += 32) {
        const int slot = a0 + lane < n_act ? m.act_slot[a0 + lane] : -1;
        const int count = slot >= 0 ? (pool.slot_rank[slot] + 7) / 8 : 0;
        int sum = count;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += y;
        }
        for (int i = 0; i < count; ++i) piece[before + sum - count + i] = make_int2(pool.slot_off[slot] + 8 * i, (a0 + lane) | i << 16);
        before += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (lane == 0) pieces = before;
    } else {
      for (int i = tid - 32; i < T * p.act; i += kBuilders - 32) table[i] = -1;
      bar_sync(kBarPairs, kBuilders - 32);
      for (int pair = tid - 32; pair < m.n; pair += kBuilders - 32) {
        const int slot = m.pair_slot[pair], tok = pair / m.J;
        // a slot named more than once by a token: its first pair stands for all
        float scale = 0.f;
        bool first = slot >= 0;
        if (first)
          for (int j = tok * m.J; j < (tok + 1) * m.J; ++j)
            if (m.pair_slot[j] == slot) first = first && j >= pair, scale += m.pair_scale[j];
        pairs[pair] = make_float2(first ? scale * pool.slot_scale[slot] : 0.f, __int_as_float(first ? pool.slot_rank[slot] : 0));
        if (first) table[tok * p.act + m.pair_act[pair]] = static_cast<int16_t>(pair);
      }
    }
    bar_sync(kBarTokens, kThreads);                   // the tokens are there (and the tables)
    const int n_pieces = pieces, units = (n_pieces + 1) / 2, own = warp - kWarps;
    constexpr int kParts = kBuilders / 32;
    float* sums = reinterpret_cast<float*>(smem + p.sum_off) + lane;
    // a few columns of B, of the CTA's first groups, to L2 while v is made
    const int first_rows = n_pieces <= kFetchPieces ? kWarps / p.split * 16 : 0;
    for (int i = tid; i < first_rows * n_pieces; i += kBuilders) {
      const int row = i / n_pieces, group = (row >> 4) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
      if (group >= F / 8) break;
      const uint16_t* b = pool.B + static_cast<size_t>((row & 8 ? F : 0) + group * 8 + (row & 7)) * pool.C + piece[i - row * n_pieces].x;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(b));
    }
    for (int u = ticket; u < units; u = ticket) {
      // 16 rows of A: a part of K to a warp
      const int2 one = piece[2 * u], two = piece[min(2 * u + 1, n_pieces - 1)];
      const uint16_t* ra = pool.A + (static_cast<size_t>(one.x) + g) * K + t * 8;
      const uint16_t* rb = pool.A + (static_cast<size_t>(two.x) + g) * K + t * 8;
      const int s0 = steps * own / kParts, s1 = steps * (own + 1) / kParts;
      clear();
      uint4 a[N], b[N];
      auto load = [&](int s, uint4& v, uint4& w) {
        const bool in = s < s1 && s * kStep + t * 8 < K;
        v = in ? __ldg(reinterpret_cast<const uint4*>(ra + s * kStep)) : make_uint4(0u, 0u, 0u, 0u);
        w = in ? __ldg(reinterpret_cast<const uint4*>(rb + s * kStep)) : make_uint4(0u, 0u, 0u, 0u);
      };
#pragma unroll
      for (int i = 0; i < N; ++i) load(s0 + i, a[i], b[i]);
      for (int s = s0; s < s1; s += N) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (s + i >= s1) break;
#pragma unroll
          for (int z = 0; z < NT; ++z) step(acc[z], a[i], b[i], x_at(z, s + i));
          load(s + i + N, a[i], b[i]);
        }
      }
#pragma unroll
      for (int z = 0; z < NT; ++z)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[(own * 4 * NT + 4 * z + i) * 32] = acc[z][i];
      bar_sync(kBarSide, kBuilders);
      if (own == 0) {
#pragma unroll
        for (int z = 0; z < NT; ++z)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = 0.f;
            for (int k = 0; k < kParts; ++k) v += sums[(k * 4 * NT + 4 * z + i) * 32];
            const int tok = 8 * z + 2 * t + (i & 1), what = i < 2 ? one.y : two.y;
            if (tok >= T || (i >= 2 && 2 * u + 1 >= n_pieces)) continue;
            const int pair = table[tok * p.act + (what & 0xffff)];
            if (pair < 0) continue;
            const int q = (what >> 16) * 8 + g;
            if (alone)
              reinterpret_cast<__nv_bfloat16*>(smem + p.v_off + pair * p.v_row)[q] = __float2bfloat16_rn(pairs[pair].x * v);
            else
              m.vpart[static_cast<size_t>(pair) * R + q] = v;
          }
        if (!alone) __threadfence();
        __syncwarp();
        if (lane == 0) {
          if (!alone) atomicAdd(&m.sync[2], 1u);
          ticket = alone ? u + 1 : static_cast<int>(atomicAdd(&m.sync[0], 1u));
        }
      }
      bar_sync(kBarSide, kBuilders);
    }
    if (n_act > 0 && !alone) {
      if (tid == 0 && units > 0) ptx::wait_counter(&m.sync[2], units, err);
      bar_sync(kBarSide, kBuilders);
      for (int i = tid; i < m.n * (R / 8); i += kBuilders) {
        const int pair = i / (R / 8), q = (i - pair * (R / 8)) * 8;
        const float c = pairs[pair].x;
        const int left = __float_as_int(pairs[pair].y) - q;               // rows of the slot from q on
        if (left <= 0) continue;
        const float4* from = reinterpret_cast<const float4*>(m.vpart + static_cast<size_t>(pair) * R + q);
        const float4 a = __ldcg(from), b = __ldcg(from + 1);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        float w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = k < left ? c * v[k] : 0.f;      // (past the rank A's rows are zero)
        *reinterpret_cast<uint4*>(smem + p.v_off + pair * p.v_row + q * 2) =
            make_uint4(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]), pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
      }
      // the last CTA leaves the counters as they were
      if (tid == 0 && atomicAdd(&m.sync[1], 1u) == gridDim.x - 1) {
        m.sync[0] = m.sync[1] = m.sync[2] = 0u;
        __threadfence();
      }
    }
    __syncthreads();                                  // v is there
    return;
  }

  // -------------------------------------------------------------------- W
  const int split = p.split, part = warp % split, each = kWarps / split, groups = F / 8;
  const int s0 = steps * part / split, s1 = steps * (part + 1) / split;
  int at = warp / split, col = 0;
  const uint16_t *gate_row = nullptr, *up_row = nullptr;
  uint4 wg[N], wu[N];
  auto load = [&](int s, uint4& a, uint4& b) {
    const bool in = s < s1 && s * kStep + t * 8 < K;
    a = in ? load_once(gate_row + s * kStep) : make_uint4(0u, 0u, 0u, 0u);
    b = in ? load_once(up_row + s * kStep) : make_uint4(0u, 0u, 0u, 0u);
  };
  auto begin = [&]() {                                // the group `at`, if there is one: its first steps
    const int i = at * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    if (i >= groups) return false;
    col = i * 8 + g;
    gate_row = W + static_cast<size_t>(col) * K + t * 8;
    up_row = W + static_cast<size_t>(F + col) * K + t * 8;
#pragma unroll
    for (int k = 0; k < N; ++k) load(s0 + k, wg[k], wu[k]);
    return true;
  };
  bool go = begin();
  ptx::grid_dependency_wait();
  // the tokens, zeros up to whole pairs of steps
  const int row_vecs = (p.x_row - 64) / 16;
  const uint32_t base = ptx::smem_u32(smem);
  for (int i = threadIdx.x; i < T * row_vecs; i += kStreamers) {
    const int tok = i / row_vecs, c = i - tok * row_vecs;
    const bool in = 8 * c < K;
    cp16(base + tok * p.x_row + c * 16, x + static_cast<size_t>(tok) * K + (in ? 8 * c : 0), in);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  bar_sync(kBarStream, kStreamers);
  bar_arrive(kBarTokens, kThreads);
  bool ready = false;
  while (go) {
    clear();
    for (int s = s0; s < s1; s += N) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (s + i >= s1) break;
#pragma unroll
        for (int z = 0; z < NT; ++z) step(acc[z], wg[i], wu[i], x_at(z, s + i));
        load(s + i + N, wg[i], wu[i]);
      }
    }
    // the side path: columns of B as further k, as many on their way
    if (!ready) __syncthreads();
    ready = true;
    const int n_pieces = pieces;
    auto bring = [&](int e, uint4& a, uint4& b) {
      const bool in = e + t < n_pieces;
      const int c = in ? piece[e + t].x : 0;
      a = in ? __ldg(reinterpret_cast<const uint4*>(pool.B + static_cast<size_t>(col) * pool.C + c)) : make_uint4(0u, 0u, 0u, 0u);
      b = in ? __ldg(reinterpret_cast<const uint4*>(pool.B + static_cast<size_t>(F + col) * pool.C + c)) : make_uint4(0u, 0u, 0u, 0u);
    };
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((part + i * split) * 4 < n_pieces) bring((part + i * split) * 4, wg[i], wu[i]);
    for (int e0 = part * 4; e0 < n_pieces; e0 += N * split * 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = e0 + i * split * 4;
        if (e >= n_pieces) break;
        const int what = e + t < n_pieces ? piece[e + t].y : -1;
#pragma unroll
        for (int z = 0; z < NT; ++z) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          const int tok = 8 * z + g;
          if (what >= 0 && tok < T) {
            const int pair = table[tok * p.act + (what & 0xffff)];
            if (pair >= 0) v = *reinterpret_cast<const uint4*>(smem + p.v_off + pair * p.v_row + (what >> 16) * 16);
          }
          step(acc[z], wg[i], wu[i], v);
        }
        if (e + N * split * 4 < n_pieces) bring(e + N * split * 4, wg[i], wu[i]);
      }
    }
    const int out = col;
    at += each;
    go = begin();                                     // the next group's first steps
    if (split > 1) {
      // the parts' sums, in order, by the group's first warp
      float* mine = reinterpret_cast<float*>(smem + p.part_off) + warp * (32 * 4 * NT) + lane;
      if (part > 0)
#pragma unroll
        for (int z = 0; z < NT; ++z)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[(4 * z + i) * 32] = acc[z][i];
      bar_sync(1 + warp / split, 32 * split);
      if (part == 0)
        for (int k = 1; k < split; ++k)
#pragma unroll
          for (int z = 0; z < NT; ++z)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[z][i] += mine[k * (32 * 4 * NT) + (4 * z + i) * 32];
      bar_sync(1 + warp / split, 32 * split);
    }
    if (part == 0) {
      auto outputs = [&](int a) {                       // one activation's code
#pragma unroll
        for (int z = 0; z < NT; ++z)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tok = 8 * z + 2 * t + i;
            if (tok < T) reinterpret_cast<__nv_bfloat16*>(h)[static_cast<size_t>(tok) * F + out] = __float2bfloat16_rn(gate(acc[z][i], a) * acc[z][2 + i]);
          }
      };
      if (act == MLORA_ACT_SILU) outputs(MLORA_ACT_SILU);
      else if (act == MLORA_ACT_GELU_TANH) outputs(MLORA_ACT_GELU_TANH);
      else outputs(MLORA_ACT_GELU);
    }
  }
  if (!ready) __syncthreads();
}

template <int NT>
cudaError_t launch_nt(const uint16_t* x, const uint16_t* W, uint16_t* h, int K, int F, int act, const PoolView& pool, const MetaView& m,
                      const StreamPlan& p, int grid, uint32_t* err, cudaStream_t s) {
  if (cudaError_t e = allow_shared_memory<gated_stream_kernel<NT>>(kStreamBytes)) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  note_launch_begin(kKindGemm, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, gated_stream_kernel<NT>, x, W, h, K, F, act, pool, m, p, err);
  note_launch_end(kKindGemm, s);
  return e;
}

}  // namespace

bool gated_streams(int T, int J, int K, int F, const PoolView& pool, int num_sms) {
  return T <= kStreamTokens && stream_plan(T, J, K, F, pool, num_sms).bytes <= kStreamBytes;
}

cudaError_t launch_gated_stream(const uint16_t* x, const uint16_t* W, uint16_t* h, int K, int F, int act, const PoolView& pool,
                                const MetaView& m, int num_sms, uint32_t* err, cudaStream_t s) {
  const StreamPlan p = stream_plan(m.T, m.J, K, F, pool, num_sms);
  // a CTA for each group or so, and for each share of the side path
  const int64_t groups = (static_cast<int64_t>(F / 8) * p.split + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(std::min<int64_t>(num_sms, std::max<int64_t>(groups, p.shares <= kOwnShares ? 0 : p.shares)));
  if (m.T <= 8) return launch_nt<1>(x, W, h, K, F, act, pool, m, p, grid, err, s);
  if (m.T <= 16) return launch_nt<2>(x, W, h, K, F, act, pool, m, p, grid, err, s);
  if (m.T <= 32) return launch_nt<4>(x, W, h, K, F, act, pool, m, p, grid, err, s);
  return launch_nt<8>(x, W, h, K, F, act, pool, m, p, grid, err, s);
}

}  // namespace mlora
