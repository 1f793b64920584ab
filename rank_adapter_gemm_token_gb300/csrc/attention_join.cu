// Joins the parts of attention items that were split among CTAs: with part k's maximum m_k (base 2), weights' sum l_k
// and weighted value sums x_k,
//     o = sum_k 2^(m_k - m) x_k / sum_k 2^(m_k - m) l_k,   m = max_k m_k,
// in an order that the split alone fixes, so the result does not depend on which CTA was first. Here the tile kernel's: the
// plan lists the split items; a unit of work is 8 rows of one, so that a few items with many parts (a chunk on a long
// context) still spread over the SMs. (The row kernel's items are joined by its own last CTAs.) Launched as a programmatic
// dependent: it reads its first task while the attention still runs. Bound by the latency of the parts' reads (from L2):
// eight parts are asked for at once. 3 to 4 us alone and cold with little to join, most of it beside the attention's end.
#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;              // rows of a unit of a tile item
constexpr int kSlices = 256 / kRows;  // units of a block

template <int HD>
__global__ void __launch_bounds__(kThreads)
attention_join_kernel(uint16_t* __restrict__ o, SeqView v) {
  constexpr int kQuads = HD / 4;       // groups of four columns
  const int units = v.counts[2] * kSlices;
  bool waited = false;
  auto wait = [&]() {
    if (!waited) ptx::grid_dependency_wait();
    waited = true;
  };
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int slice = u % kSlices, w = slice / (kSlices / 2);
    const int4 task = *reinterpret_cast<const int4*>(v.tile_join + u / kSlices);
    const TileBlk b = v.blk[task.x];
    const int kvh = task.y, parts = task.w;
    const int r = slice % (kSlices / 2) * kRows + static_cast<int>(threadIdx.x) % kRows, quad = static_cast<int>(threadIdx.x) / kRows;
    const int tok = b.t0 + v.tile_tokens * w + r / v.G;
    if (quad >= kQuads || r >= v.tile_tokens * v.G || tok >= b.n) continue;
    const int64_t slot = tile_slot(v);
    const float* base = v.tile_part + (4 * static_cast<int64_t>(task.z) + w) * slot;    // part k > 0: base + 4 k slot
    wait();
    Sums z{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = 0; k0 < parts; k0 += kPartsAhead) {
      float m[kPartsAhead], l[kPartsAhead];
      float4 y[kPartsAhead];
#pragma unroll
      for (int k = 0; k < kPartsAhead; ++k) {
        const int part = min(k0 + k, parts - 1);
        const float* p = base + (part == 0 ? 2 * slot : 4 * part * slot);
        m[k] = __ldcg(p + 128 * HD + r);
        l[k] = __ldcg(p + 128 * HD + 128 + r);
        y[k] = __ldcg(reinterpret_cast<const float4*>(p) + quad * 128 + r);
      }
#pragma unroll
      for (int k = 0; k < kPartsAhead; ++k)
        if (k0 + k < parts) z.add(m[k], l[k], y[k]);
    }
    const float inv = inverse(z.total);
    *reinterpret_cast<uint2*>(o + (static_cast<int64_t>(b.start + tok) * v.Hq + kvh * v.G + r % v.G) * HD + 4 * quad) =
        make_uint2(pack_bf16(z.x.x * inv, z.x.y * inv), pack_bf16(z.x.z * inv, z.x.w * inv));
  }
  wait();                              // the grid's end stands for the end of the attention
}

}  // namespace

cudaError_t launch_attention_join(uint16_t* o, const SeqView& s, cudaStream_t st) {
  note_launch_begin(kKindAttn, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(4 * s.tile_ctas);
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
