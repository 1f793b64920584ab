// Joins the parts of attention items that were split among CTAs: with part k's maximum m_k (base 2), weights' sum l_k
// and weighted value sums x_k,
//     o = sum_k 2^(m_k - m) x_k / sum_k 2^(m_k - m) l_k,   m = max_k m_k,
// in an order that the split alone fixes, so the result does not depend on which CTA was first. The plan lists the split
// items; a unit of work is a row item whole, or 8 rows of a tile item, so that a few items with many parts (a chunk on a
// long context) still spread over the SMs. Launched as a programmatic dependent: it reads its first task while the
// attention still runs. Bound by the latency of the parts' reads (from L2): eight parts are asked for at once, and where a
// row item has fewer elements than the CTA threads, its parts are divided among groups of threads. Measured alone and cold:
// 4 us with nothing to join, 7 to 10 for the 304 to 456 cuts of 128 sequences; most of it overlaps the attention's end.
#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;              // rows of a unit of a tile item
constexpr int kSlices = 256 / kRows;  // units of a block
constexpr int kAhead = 8;             // parts asked for at once

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse(float total) {
  return total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;      // an empty row is zero; NaN stays
}

// Running maximum, sum of weights and four weighted value sums.
struct Sums {
  float top, total;
  float4 x;
  __device__ __forceinline__ void add(float m, float l, const float4& y) {
    if (m == -INFINITY) return;       // (a part that saw none of the row's keys has no sums)
    const float up = fmaxf(top, m);
    const float f = exp2_approx(top - up), g = exp2_approx(m - up);
    top = up;
    total = total * f + l * g;
    x.x = x.x * f + y.x * g;
    x.y = x.y * f + y.y * g;
    x.z = x.z * f + y.z * g;
    x.w = x.w * f + y.w * g;
  }
};

template <int HD>
__global__ void __launch_bounds__(kThreads)
attention_join_kernel(uint16_t* __restrict__ o, SeqView v) {
  constexpr int kQuads = HD / 4;       // groups of four columns
  __shared__ float4 sx[kThreads];
  __shared__ float2 sm[kThreads];
  const int row_units = v.counts[2], units = row_units + v.counts[3] * kSlices;
  bool waited = false;
  auto wait = [&]() {
    if (!waited) ptx::grid_dependency_wait();
    waited = true;
  };
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    if (u < row_units) {
      const int4 task = *reinterpret_cast<const int4*>(v.row_join + u);
      const int4 sq = *reinterpret_cast<const int4*>(v.row_seq + task.x);
      const int kvh = task.y, parts = task.w, elements = sq.y * v.G * kQuads;
      const int64_t slot = row_slot(v);
      const float* base = v.row_part + 2 * static_cast<int64_t>(task.z) * slot;      // part k > 0: base + 2 k slot
      wait();
      // threads beyond the elements take a share of the parts
      const int groups = max(1, kThreads / elements);
      for (int i0 = 0; i0 < elements; i0 += kThreads) {
        const int e = groups > 1 ? static_cast<int>(threadIdx.x) % elements : i0 + static_cast<int>(threadIdx.x);
        const int g = groups > 1 ? static_cast<int>(threadIdx.x) / elements : 0;
        const bool mine = e < elements && g < groups;
        const int r = mine ? e / kQuads : 0, h = e % kQuads * 4;
        Sums z{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        if (mine) {
          for (int k0 = g; k0 < parts; k0 += kAhead * groups) {
            float2 ml[kAhead];
            float4 y[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              const int part = min(k0 + k * groups, parts - 1);
              const float* p = base + (part == 0 ? slot : 2 * part * slot);
              ml[k] = __ldcg(reinterpret_cast<const float2*>(p + v.row_limit * HD + 2 * r));
              y[k] = __ldcg(reinterpret_cast<const float4*>(p + r * HD + h));
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
              if (k0 + k * groups < parts) z.add(ml[k].x, ml[k].y, y[k]);
          }
        }
        if (groups > 1) {
          sm[threadIdx.x] = make_float2(z.top, z.total);
          sx[threadIdx.x] = z.x;
          __syncthreads();
          if (mine && g == 0)
            for (int k = 1; k < groups; ++k) {
              const float2 ml = sm[threadIdx.x + k * elements];
              z.add(ml.x, ml.y, sx[threadIdx.x + k * elements]);
            }
          __syncthreads();
        }
        if (mine && g == 0) {
          const float inv = inverse(z.total);
          *reinterpret_cast<uint2*>(o + (static_cast<int64_t>(sq.w + r / v.G) * v.Hq + kvh * v.G + r % v.G) * HD + h) =
              make_uint2(pack_bf16(z.x.x * inv, z.x.y * inv), pack_bf16(z.x.z * inv, z.x.w * inv));
        }
      }
      continue;
    }
    const int unit = u - row_units, slice = unit % kSlices, w = slice / (kSlices / 2);
    const int4 task = *reinterpret_cast<const int4*>(v.tile_join + unit / kSlices);
    const TileBlk b = v.blk[task.x];
    const int kvh = task.y, parts = task.w;
    const int r = slice % (kSlices / 2) * kRows + static_cast<int>(threadIdx.x) % kRows, quad = static_cast<int>(threadIdx.x) / kRows;
    const int tok = b.t0 + v.tile_tokens * w + r / v.G;
    if (quad >= kQuads || r >= v.tile_tokens * v.G || tok >= b.n) continue;
    const int64_t slot = tile_slot(v);
    const float* base = v.tile_part + (4 * static_cast<int64_t>(task.z) + w) * slot;    // part k > 0: base + 4 k slot
    wait();
    Sums z{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = 0; k0 < parts; k0 += kAhead) {
      float m[kAhead], l[kAhead];
      float4 y[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int part = min(k0 + k, parts - 1);
        const float* p = base + (part == 0 ? 2 * slot : 4 * part * slot);
        m[k] = __ldcg(p + 128 * HD + r);
        l[k] = __ldcg(p + 128 * HD + 128 + r);
        y[k] = __ldcg(reinterpret_cast<const float4*>(p) + quad * 128 + r);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k0 + k < parts) z.add(m[k], l[k], y[k]);
    }
    const float inv = inverse(z.total);
    *reinterpret_cast<uint2*>(o + (static_cast<int64_t>(b.start + tok) * v.Hq + kvh * v.G + r % v.G) * HD + 4 * quad) =
        make_uint2(pack_bf16(z.x.x * inv, z.x.y * inv), pack_bf16(z.x.z * inv, z.x.w * inv));
  }
  wait();                              // the grid's end stands for the end of the attention
}

}  // namespace

cudaError_t launch_attention_join(uint16_t* o, const SeqView& s, bool tiles, cudaStream_t st) {
  note_launch_begin(kKindAttn, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((tiles ? 4 : 2) * s.tile_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = s.hd == 128 ? cudaLaunchKernelEx(&cfg, attention_join_kernel<128>, o, s)
                                    : cudaLaunchKernelEx(&cfg, attention_join_kernel<64>, o, s);
  note_launch_end(kKindAttn, st);
  return e;
}

}  // namespace mlora
