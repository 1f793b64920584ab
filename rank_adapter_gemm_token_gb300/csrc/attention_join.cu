// Joins the parts of attention items that were split among CTAs: with part k's maximum m_k (base 2), weights' sum l_k
// and weighted value sums x_k,
//     o = sum_k 2^(m_k - m) x_k / sum_k 2^(m_k - m) l_k,   m = max_k m_k,
// in the order of the keys, so the result does not depend on which CTA was first. A CTA for each cut that may be the
// first inside an item (most leave at once): a row item whole, a tile item in slices of 32 rows. Launched as a
// programmatic dependent: it reads its task while the attention still runs. Bound by the latency of two dependent
// reads of the L2, where the parts still are.
#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kThreads = 128;
constexpr int kSlices = 8;            // of a block

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse(float total) {
  return total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;      // an empty row is zero; NaN stays
}

template <int HD>
__global__ void __launch_bounds__(kThreads)
attention_join_kernel(uint16_t* __restrict__ o, SeqView v) {
  const bool row = static_cast<int>(blockIdx.x) < v.row_ctas;
  const int idx = static_cast<int>(blockIdx.x) - (row ? 0 : v.row_ctas);
  const int4 task = *reinterpret_cast<const int4*>(row ? v.row_join + idx : v.tile_join + idx / kSlices);
  const int kvh = task.y, cta = task.z, parts = task.w;
  if (parts == 0) {                     // (the grid's end stands for the end of the attention: every CTA waits for it)
    ptx::grid_dependency_wait();
    return;
  }
  if (row) {
    const int4 sq = *reinterpret_cast<const int4*>(v.row_seq + task.x);
    const int rows = sq.y * v.G;
    const int64_t slot = row_slot(v);
    const float* first = v.row_part + (2 * static_cast<int64_t>(cta) + 1) * slot;           // part 0; part k: CTA cta + k
    auto part = [&](int k) { return k == 0 ? first : v.row_part + 2 * static_cast<int64_t>(cta + k) * slot; };
    ptx::grid_dependency_wait();
    for (int i = threadIdx.x; i < rows * (HD / 4); i += kThreads) {
      const int r = i / (HD / 4), h = i % (HD / 4) * 4;
      float top = -INFINITY, total = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kAhead = 8;
      for (int k0 = 0; k0 < parts; k0 += kAhead) {
        float2 ml[kAhead];
        float4 y[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float* p = part(min(k0 + k, parts - 1));
          ml[k] = __ldcg(reinterpret_cast<const float2*>(p + v.row_limit * HD + 2 * r));
          y[k] = __ldcg(reinterpret_cast<const float4*>(p + r * HD + h));
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (k0 + k >= parts || ml[k].x == -INFINITY) continue;
          const float up = fmaxf(top, ml[k].x);
          const float f = exp2_approx(top - up), g = exp2_approx(ml[k].x - up);
          top = up;
          total = total * f + ml[k].y * g;
          x.x = x.x * f + y[k].x * g;
          x.y = x.y * f + y[k].y * g;
          x.z = x.z * f + y[k].z * g;
          x.w = x.w * f + y[k].w * g;
        }
      }
      const float inv = inverse(total);
      *reinterpret_cast<uint2*>(o + (static_cast<int64_t>(sq.w + r / v.G) * v.Hq + kvh * v.G + r % v.G) * HD + h) =
          make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    }
    return;
  }
  const TileBlk b = v.blk[task.x];
  const int slice = idx % kSlices, w = slice / 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tr = (slice & 3) * 32 + lane, tok = b.t0 + v.tile_tokens * w + tr / v.G;
  const bool valid = tr < v.tile_tokens * v.G && tok < b.n;
  const int64_t slot = tile_slot(v);
  auto part = [&](int k) { return v.tile_part + ((2 * static_cast<int64_t>(cta + k) + (k == 0)) * 2 + w) * slot; };
  ptx::grid_dependency_wait();
  if (!__any_sync(0xffffffffu, valid)) return;
  float top = -INFINITY, total = 0.f;
  for (int k0 = 0; k0 < parts; k0 += 4) {
    float m[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float* p = part(min(k0 + k, parts - 1)) + 128 * HD + tr;
      m[k] = __ldcg(p);
      l[k] = __ldcg(p + 128);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k0 + k >= parts || m[k] == -INFINITY) continue;
      const float up = fmaxf(top, m[k]);
      total = total * exp2_approx(top - up) + l[k] * exp2_approx(m[k] - up);
      top = up;
    }
  }
  const float inv = inverse(total);
  constexpr int kCols = HD / 16;                       // four-column groups of a warp: groups warp, warp + 4, ...
  float4 x[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const float* p = part(k);
    const float m = __ldcg(p + 128 * HD + tr);
    float4 y[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) y[c] = __ldcg(reinterpret_cast<const float4*>(p) + (warp + 4 * c) * 128 + tr);
    if (m == -INFINITY) continue;                      // (a part that saw none of the row's keys has no sums)
    const float f = exp2_approx(m - top) * inv;
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      x[c].x = fmaf(f, y[c].x, x[c].x);
      x[c].y = fmaf(f, y[c].y, x[c].y);
      x[c].z = fmaf(f, y[c].z, x[c].z);
      x[c].w = fmaf(f, y[c].w, x[c].w);
    }
  }
  if (!valid) return;
  uint16_t* dst = o + (static_cast<int64_t>(b.start + tok) * v.Hq + kvh * v.G + tr % v.G) * HD;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    *reinterpret_cast<uint2*>(dst + 4 * (warp + 4 * c)) = make_uint2(pack_bf16(x[c].x, x[c].y), pack_bf16(x[c].z, x[c].w));
}

}  // namespace

cudaError_t launch_attention_join(uint16_t* o, const SeqView& s, bool tiles, cudaStream_t st) {
  note_launch_begin(kKindAttn, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(s.row_ctas + (tiles ? s.tile_ctas * kSlices : 0));
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
