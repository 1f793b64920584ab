// The paged cache's own kernels.
//
// qkv_write: a step's qkv rows (the qkv linear's fp32 output) on their way to the attention. For each
// token and head of hd elements x:
//     x <- x / sqrt(mean(x^2) + eps) * w                        queries and keys, where a weight is given
//     (a, b) <- m (a cos - b sin, b cos + a sin)                 queries and keys, the first rot elements
//     queries: bf16 row of q; keys and values: row pos % page of page table[pos / page], as bf16 or as
//     e4m3 codes rn(x / s) with s = max(max |x|, 2^-60) / 448, one fp32 s for each token and head.
// A row with an infinity or a NaN gets codes 0 and the scale NaN, so that all of it reads back as NaN.
// Angles are taken in turns: pos * f with f a sum of two floats, the whole turns dropped exactly
// (product and its rounding error by fma), then sin and cos of the fraction: about 1e-7 for every
// position up to 2^24, where an fp32 angle in radians would be off by pos * 6e-8.
// Bound: HBM, each value read once and written once; a warp holds whole heads in registers (a lane hd / 32
// adjacent elements), so that norm, rotation and maximum are shuffles.
//
// kv_read: whole sequences' cached rows as dense bf16 rows [token, head, hd]; a copy (bf16) or code * scale
// rounded once (e4m3). Bound: HBM.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kWriteWarps = 8;

template <int V>
struct Vec;
template <>
struct Vec<4> {
  static __device__ __forceinline__ void load(const float* p, float* x) {
    const float4 f = __ldcs(reinterpret_cast<const float4*>(p));
    x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
  }
  static __device__ __forceinline__ void store_bf16(uint16_t* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
  static __device__ __forceinline__ void store_e4m3(uint8_t* p, const float* x) {
    *reinterpret_cast<uint32_t*>(p) = pack_e4m3(x[0], x[1]) | (pack_e4m3(x[2], x[3]) << 16);
  }
};
template <>
struct Vec<2> {
  static __device__ __forceinline__ void load(const float* p, float* x) {
    const float2 f = __ldcs(reinterpret_cast<const float2*>(p));
    x[0] = f.x, x[1] = f.y;
  }
  static __device__ __forceinline__ void store_bf16(uint16_t* p, const float* x) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(x[0], x[1]);
  }
  static __device__ __forceinline__ void store_e4m3(uint8_t* p, const float* x) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(pack_e4m3(x[0], x[1]));
  }
};

// A warp: up to HPW consecutive heads of one token (heads: the query heads, the key heads, the value heads).
template <int HD, int HPW>
__global__ void __launch_bounds__(kWriteWarps * 32)
qkv_write_kernel(const float* __restrict__ qkv, int64_t ld, const uint16_t* __restrict__ q_norm,
                 const uint16_t* __restrict__ k_norm, float eps, RopeView rope, const int32_t* __restrict__ positions,
                 uint16_t* __restrict__ q, KvView kv, SeqView s) {
  constexpr int V = HD / 32;
  const int lane = threadIdx.x & 31;
  const int heads = s.Hq + 2 * s.Hkv;
  const int groups = (heads + HPW - 1) / HPW;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWriteWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / groups), h0 = static_cast<int>(w % groups) * HPW;
  if (t >= s.T) return;
  const int e = lane * V;
  float x[HPW][V];
#pragma unroll
  for (int i = 0; i < HPW; ++i)
    if (h0 + i < heads) Vec<V>::load(qkv + t * ld + static_cast<int64_t>(h0 + i) * HD + e, x[i]);
  const int row = s.tok_row[t];
  const bool none = s.tok_seq[t] < 0;

  // this lane's angles (the same for every head of the token)
  float cs[V], sn[V];
  int from = lane;                       // lane holding the other elements of this lane's pairs
  bool turned = false, second = false;
  if (rope.rot > 0 && h0 < s.Hq + s.Hkv) {
    const int half = rope.rot >> 1;
    turned = e < rope.rot;
    second = !rope.interleaved && e >= half;
    from = (!turned || rope.interleaved) ? lane : second ? lane - half / V : lane + half / V;
    const float pos = static_cast<float>(positions ? positions[t] : s.tok_pos[t]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = !turned ? 0 : rope.interleaved ? (e + j) >> 1 : second ? e + j - half : e + j;
      const float2 f = __ldg(rope.freq + i);
      const float p = pos * f.x;
      float frac = p - rintf(p);
      frac += fmaf(pos, f.x, -p) + pos * f.y;
      sincospif(2.0f * frac, &sn[j], &cs[j]);
      sn[j] *= rope.mscale;
      cs[j] *= rope.mscale;
    }
  }

#pragma unroll
  for (int i = 0; i < HPW; ++i) {
    const int h = h0 + i;
    if (h >= heads) break;
    const bool is_q = h < s.Hq, is_k = !is_q && h < s.Hq + s.Hkv;
    const uint16_t* norm = is_q ? q_norm : is_k ? k_norm : nullptr;
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) sum = fmaf(x[i][j], x[i][j], sum);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      const float r = 1.0f / sqrtf(sum * (1.0f / HD) + eps);
#pragma unroll
      for (int j = 0; j < V; ++j) x[i][j] *= r * __uint_as_float(static_cast<uint32_t>(__ldg(norm + e + j)) << 16);
    }
    if ((is_q || is_k) && rope.rot > 0) {
      if (rope.interleaved) {
        if (turned) {
#pragma unroll
          for (int j = 0; j < V; j += 2) {
            const float a = x[i][j], b = x[i][j + 1];
            x[i][j] = a * cs[j] - b * sn[j];
            x[i][j + 1] = b * cs[j] + a * sn[j];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float other = __shfl_sync(0xffffffffu, x[i][j], from);
          if (turned) x[i][j] = second ? x[i][j] * cs[j] + other * sn[j] : x[i][j] * cs[j] - other * sn[j];
        }
      }
    }
    if (is_q) {
      if (none) {
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][j] = 0.f;
      }
      Vec<V>::store_bf16(q + (static_cast<int64_t>(t) * s.Hq + h) * HD + e, x[i]);
      continue;
    }
    if (row < 0) continue;
    const int kh = is_k ? h - s.Hq : h - s.Hq - s.Hkv;
    const int64_t at = ((static_cast<int64_t>(row >> kv.page_log2) * kv.Hkv + kh) << kv.page_log2) + (row & (kv.page - 1));
    void* base = is_k ? kv.K : kv.V;
    if (kv.type == kKvBf16) {
      Vec<V>::store_bf16(static_cast<uint16_t*>(base) + at * HD + e, x[i]);
      continue;
    }
    float most = 0.f;
    bool finite = true;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      most = fmaxf(most, fabsf(x[i][j]));
      finite = finite && fabsf(x[i][j]) <= 3.402823466e38f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    finite = __all_sync(0xffffffffu, finite);
    const float scale = finite ? fmaxf(most, kAmaxMin) / kE4m3Max : __int_as_float(0x7fffffff);
    const float inv = 1.0f / scale;
#pragma unroll
    for (int j = 0; j < V; ++j) x[i][j] = finite ? x[i][j] * inv : 0.f;
    Vec<V>::store_e4m3(static_cast<uint8_t*>(base) + at * HD + e, x[i]);
    if (lane == 0) (is_k ? kv.k_scale : kv.v_scale)[at] = scale;
  }
}

constexpr int kReadWarps = 8;

// A warp: one head of one cached page, K and V, 16 bytes of output row per lane and step.
template <int HD, bool E4M3>
__global__ void __launch_bounds__(kReadWarps * 32)
kv_read_kernel(const int32_t* __restrict__ row_start, int64_t rows, uint16_t* __restrict__ k_out,
               uint16_t* __restrict__ v_out, KvView kv, SeqView s) {
  constexpr int kLanes = HD / 8;                          // lanes of one row (8 elements each)
  constexpr int kRows = 32 / kLanes;                      // rows of one step
  const int lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(s.page_pre[s.S]) * kv.Hkv;
  const int e = (lane % kLanes) * 8, r0 = lane / kLanes;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5); w < units;
       w += static_cast<int64_t>(gridDim.x) * kReadWarps) {
    const int g = static_cast<int>(w / kv.Hkv), h = static_cast<int>(w - static_cast<int64_t>(g) * kv.Hkv);
    const int sq = last_at_most(s.page_pre, s.S, g);
    const int pi = g - s.page_pre[sq];
    const int cnt = min(kv.page, s.len[sq] - (pi << kv.page_log2));
    const int64_t dst = static_cast<int64_t>(row_start[sq]) + (static_cast<int64_t>(pi) << kv.page_log2);
    if (dst < 0 || dst + cnt > rows) {
      if (lane == 0) atomicOr(s.err, ptx::kErrBadRow);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(s.table[static_cast<size_t>(sq) * s.max_pages + pi]) * kv.Hkv + h) << kv.page_log2;
#pragma unroll 4
    for (int r = r0; r < cnt; r += kRows) {
      const int64_t to = ((dst + r) * kv.Hkv + h) * HD + e;
      if (E4M3) {
        const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.K) + (at + r) * HD + e);
        const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.V) + (at + r) * HD + e);
        *reinterpret_cast<uint4*>(k_out + to) = e4m3_times(a, kv.k_scale[at + r]);
        *reinterpret_cast<uint4*>(v_out + to) = e4m3_times(b, kv.v_scale[at + r]);
      } else {
        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv.K) + (at + r) * HD + e);
        const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv.V) + (at + r) * HD + e);
        *reinterpret_cast<uint4*>(k_out + to) = a;
        *reinterpret_cast<uint4*>(v_out + to) = b;
      }
    }
  }
}

template <int HD, int HPW>
cudaError_t write_as(const float* qkv, int64_t ld, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                     const RopeView& rope, const int32_t* positions, uint16_t* q, const KvView& kv, const SeqView& s,
                     cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(s.T) * ((s.Hq + 2 * s.Hkv + HPW - 1) / HPW);
  const int grid = static_cast<int>((warps + kWriteWarps - 1) / kWriteWarps);
  note_launch_begin(kKindKv, st);
  qkv_write_kernel<HD, HPW><<<grid, kWriteWarps * 32, 0, st>>>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s);
  const cudaError_t e = cudaGetLastError();
  note_launch_end(kKindKv, st);
  return e;
}

}  // namespace

cudaError_t launch_qkv_write(const float* qkv, int64_t ld, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                             const RopeView& rope, const int32_t* positions, uint16_t* q, const KvView& kv,
                             const SeqView& s, int num_sms, cudaStream_t st) {
  if (s.T == 0) return cudaSuccess;
  // One head per warp while that leaves SMs without a full set of warps, else four: the angles are
  // made once per warp and token.
  const bool few = static_cast<int64_t>(s.T) * (s.Hq + 2 * s.Hkv) < 64L * num_sms;
  if (s.hd == 128)
    return few ? write_as<128, 1>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st)
               : write_as<128, 4>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st);
  return few ? write_as<64, 1>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st)
             : write_as<64, 4>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st);
}

cudaError_t launch_kv_read(const int32_t* row_start, int64_t rows, uint16_t* k, uint16_t* v, const KvView& kv,
                           const SeqView& s, int num_sms, cudaStream_t st) {
  if (s.S == 0) return cudaSuccess;
  const int64_t most = std::max<int64_t>(1, (rows / kv.page + s.S) * kv.Hkv);      // units of a call that fits
  const int grid = static_cast<int>(std::min<int64_t>((most + kReadWarps - 1) / kReadWarps, 8L * num_sms));
  note_launch_begin(kKindKv, st);
  if (kv.hd == 128) {
    if (kv.type == kKvE4m3)
      kv_read_kernel<128, true><<<grid, kReadWarps * 32, 0, st>>>(row_start, rows, k, v, kv, s);
    else
      kv_read_kernel<128, false><<<grid, kReadWarps * 32, 0, st>>>(row_start, rows, k, v, kv, s);
  } else {
    if (kv.type == kKvE4m3)
      kv_read_kernel<64, true><<<grid, kReadWarps * 32, 0, st>>>(row_start, rows, k, v, kv, s);
    else
      kv_read_kernel<64, false><<<grid, kReadWarps * 32, 0, st>>>(row_start, rows, k, v, kv, s);
  }
  const cudaError_t e = cudaGetLastError();
  note_launch_end(kKindKv, st);
  return e;
}

}  // namespace mlora
