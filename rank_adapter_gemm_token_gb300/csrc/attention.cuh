// Device helpers shared by the attention step's kernels: 16-bit and e4m3 packing, and the searches
// over a step's prefix sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace mlora {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (low byte: lo), round to nearest even, saturating.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four e4m3 codes as two pairs of halves: exact, every e4m3 value is an f16 value. (Both halves of the register are named, so
// that the upper one needs no shift.)
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// 32 bytes, in one store where the output is 32-byte aligned.
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t* x, bool wide) {
  if (!wide) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}
// Eight e4m3 codes times a scale, as bf16 (each product rounded to fp32, then to bf16).
__device__ __forceinline__ uint4 e4m3_times(uint2 c, float scale) {
  uint4 out;
  uint32_t h[4];
  e4m3x4_f16x4(c.x, h[0], h[1]);
  e4m3x4_f16x4(c.y, h[2], h[3]);
  uint32_t* o = &out.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    o[i] = pack_bf16(f.x * scale, f.y * scale);
  }
  return out;
}

// The last i in [0, n) with pre[i] <= x, for ascending prefix sums with pre[0] <= x (one warp, all lanes).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* pre, int n, T x) {
  int lo = 0, len = n;                                   // the answer lies in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + min(static_cast<int>(threadIdx.x & 31) * step, len - 1);
    const uint32_t below = __ballot_sync(0xffffffffu, pre[at] <= x);
    const int next = min((31 - __clz(below | 1u)) * step, len - 1);
    len = min(step, len - next);
    lo += next;
  }
  return lo;
}

// An equal share of a list of work items for each of n CTAs. The items' units (keys of 64 or 128) lie one
// after another, total in all; CTA c takes units [cut(c), cut(c + 1)), so an item that lies across a cut
// is split and its parts are joined. An item's first `head` units stand for its fixed costs, the others for
// its keys. A cut in the head, or within `snap` units of the keys' ends, moves to the item's end, and any cut in an item too
// short for others moves to the nearer end: a split costs more than that imbalance.
struct Shares {
  int64_t total;
  int n;
  int head, snap;
  __device__ __forceinline__ int64_t raw(int64_t c) const { return total * c / n; }
  // cut(c) when it falls into the item of units [a, b)
  __device__ __forceinline__ int64_t snapped(int64_t x, int64_t a, int64_t b) const {
    const int64_t lo = a + head + snap + 1, hi = b - snap - 1;
    if (lo > hi) return 2 * (x - a) <= b - a ? a : b;
    return x < lo ? a : x > hi ? b : x;
  }
  // The cuts that split the item [a, b): CTAs first + 1 ... first + count begin inside it.
  __device__ __forceinline__ void inside(int64_t a, int64_t b, int* first, int* count) const {
    const int64_t lo = a + head + snap + 1, hi = b - snap - 1;      // raw cuts in [lo, hi] stay inside
    if (lo > hi) {
      *first = 0, *count = 0;
      return;
    }
    const int64_t c0 = (lo * n + total - 1) / total;          // least c with raw(c) >= lo
    const int64_t c1 = ((hi + 1) * n - 1) / total;            // largest c with raw(c) <= hi
    *first = static_cast<int>(c0) - 1;
    *count = static_cast<int>(c1 >= c0 ? c1 - c0 + 1 : 0);
  }
};

}  // namespace mlora
