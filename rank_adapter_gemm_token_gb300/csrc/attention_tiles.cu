// Attention of sequences with many query rows (chunks of a prompt, whole prompts) over the paged cache, the
// formula of attention_rows.cu. A warp for each row, keys one after another: right for every case, and slow.
#include <algorithm>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kThreads = 256;

template <int HD, bool E4M3>
__device__ __forceinline__ void load_row(const void* base, int64_t at, int lane, float* x) {
  constexpr int V = HD / 32;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t i = at * HD + lane * V + j;
    if (E4M3) {
      const uint32_t h = e4m3x2_f16x2(static_cast<const uint8_t*>(base)[i]);
      x[j] = __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
    } else {
      x[j] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
    }
  }
}

template <int HD, bool E4M3>
__global__ void __launch_bounds__(kThreads)
attention_tiles_kernel(const uint16_t* __restrict__ q, uint16_t* __restrict__ o, float scale_log2, KvView kv, SeqView v) {
  constexpr int V = HD / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = v.counts[0];
  for (int item = blockIdx.x; item < blocks * v.Hkv; item += gridDim.x) {
    const int j = item / v.Hkv, kvh = item % v.Hkv;
    const int s = v.blk_seq[j], r0 = v.blk_row[j];
    const int n = v.n[s], len = v.len[s], first = v.start[s];
    const int32_t* table = v.table + static_cast<size_t>(s) * v.max_pages;
    for (int r = r0 + warp; r < min(r0 + kBlockRows, n * v.G); r += kThreads / 32) {
      const int64_t row = (static_cast<int64_t>(first + r / v.G) * v.Hq + kvh * v.G + r % v.G) * HD;
      float x[V], acc[V], m = -INFINITY, l = 0.f;
#pragma unroll
      for (int k = 0; k < V; ++k) x[k] = __uint_as_float(static_cast<uint32_t>(q[row + lane * V + k]) << 16), acc[k] = 0.f;
      for (int key = 0; key <= len - n + r / v.G; ++key) {
        const int64_t at = ((static_cast<int64_t>(table[key >> kv.page_log2]) * v.Hkv + kvh) << kv.page_log2) + (key & (kv.page - 1));
        float y[V], d = 0.f;
        load_row<HD, E4M3>(kv.K, at, lane, y);
#pragma unroll
        for (int k = 0; k < V; ++k) d = fmaf(x[k], y[k], d);
#pragma unroll
        for (int b = 16; b > 0; b >>= 1) d += __shfl_xor_sync(0xffffffffu, d, b);
        if (E4M3) d *= kv.k_scale[at];
        d *= scale_log2;
        const float top = fmaxf(m, d), f = top == m ? 1.f : exp2f(m - top), p = exp2f(d - top);
        m = top;
        l = l * f + p;
        load_row<HD, E4M3>(kv.V, at, lane, y);
        const float vs = E4M3 ? kv.v_scale[at] : 1.f;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = fmaf(p * vs, y[k], acc[k] * f);
      }
#pragma unroll
      for (int k = 0; k < V; ++k) o[row + lane * V + k] = static_cast<uint16_t>(pack_bf16(acc[k] / l, 0.f));
    }
  }
}

}  // namespace

cudaError_t launch_attention_tiles(const uint16_t* q, uint16_t* o, float scale, const KvView& kv, const SeqView& s,
                                   cudaStream_t st) {
  const float c = scale * 1.4426950408889634f;
  const int grid = s.tile_ctas * 8;
  note_launch_begin(kKindAttn, st);
  if (s.hd == 128) {
    if (kv.type == kKvE4m3) attention_tiles_kernel<128, true><<<grid, kThreads, 0, st>>>(q, o, c, kv, s);
    else attention_tiles_kernel<128, false><<<grid, kThreads, 0, st>>>(q, o, c, kv, s);
  } else {
    if (kv.type == kKvE4m3) attention_tiles_kernel<64, true><<<grid, kThreads, 0, st>>>(q, o, c, kv, s);
    else attention_tiles_kernel<64, false><<<grid, kThreads, 0, st>>>(q, o, c, kv, s);
  }
  const cudaError_t e = cudaGetLastError();
  note_launch_end(kKindAttn, st);
  return e;
}

}  // namespace mlora
