// h = act(g) * u from the fp32 rows [g u] of the stacked gate and up projections.
//
// Bound: HBM or L2, 10 bytes an output (8 read, 2 written). A thread takes 8 outputs of a row: two 32-byte reads each of the
// gate's and the up projection's columns, one 16-byte store.
#include <algorithm>

#include "attention.cuh"
#include "gated.cuh"
#include "internal.h"

namespace mlora {
namespace {

constexpr int kThreads = 256;

template <int ACT>
__global__ void __launch_bounds__(kThreads)
gated_activation_kernel(const float* __restrict__ y, uint16_t* __restrict__ h, int64_t groups, int row_groups) {
  const int F = 8 * row_groups;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < groups; i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t row = i / row_groups;
    const float* g = y + row * 2 * F + (i - row * row_groups) * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 a = reinterpret_cast<const float4*>(g)[k], b = reinterpret_cast<const float4*>(g + F)[k];
      v[4 * k] = gate(a.x, ACT) * b.x, v[4 * k + 1] = gate(a.y, ACT) * b.y;
      v[4 * k + 2] = gate(a.z, ACT) * b.z, v[4 * k + 3] = gate(a.w, ACT) * b.w;
    }
    reinterpret_cast<uint4*>(h)[i] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
}

}  // namespace

cudaError_t launch_gated_activation(const float* y, uint16_t* h, int T, int F, int act, int num_sms, cudaStream_t s) {
  const int64_t groups = static_cast<int64_t>(T) * (F / 8);
  if (groups == 0) return cudaSuccess;
  const int blocks = static_cast<int>(std::min<int64_t>((groups + kThreads - 1) / kThreads, 8LL * num_sms));
  note_launch_begin(kKindAct, s);
  const auto kernel = act == MLORA_ACT_SILU        ? gated_activation_kernel<MLORA_ACT_SILU>
                      : act == MLORA_ACT_GELU_TANH ? gated_activation_kernel<MLORA_ACT_GELU_TANH>
                                                   : gated_activation_kernel<MLORA_ACT_GELU>;
  kernel<<<blocks, kThreads, 0, s>>>(y, h, groups, F / 8);
  const cudaError_t e = cudaGetLastError();
  note_launch_end(kKindAct, s);
  return e;
}

}  // namespace mlora
