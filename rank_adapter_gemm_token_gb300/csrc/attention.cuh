// Device helpers shared by the attention step's kernels: 16-bit and e4m3 packing, and the searches
// over a step's prefix sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "attention.h"
#include "per_device.h"

namespace mlora {

// Allows a kernel's launches on the current device this many bytes of dynamic shared memory.
template <auto Kernel>
cudaError_t allow_shared_memory(int bytes) {
  static std::atomic<uint64_t> done{0};
  int device = 0;
  if (cudaError_t e = cudaGetDevice(&device)) return e;
  return once_per_device<cudaError_t>(done, device, [&] {
    return cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
}

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

// Query rows in f16: the power of two that lifts a row whose largest magnitude is `most` (bf16) to [2^14, 2^15), and its
// inverse. bf16 numbers stay exact down to 2^-31 of the row's largest. (Rows below 2^-112 are lifted by 2^126, the largest
// power whose inverse is a normal number.)
__device__ __forceinline__ float query_lift(float most, float* back) {
  const int e = __float_as_int(most) >> 23;              // biased; 0 for subnormal numbers and 0
  *back = __int_as_float(max(1, e - 14) << 23);
  return __int_as_float(min(253, 268 - e) << 23);
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

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Joining the parts of split attention items.
constexpr int kPartsAhead = 8;           // parts asked for at once
// The inverse of a row's sum of weights. Every row that is written sees a key, its own: a sum of 0 is that of scores that
// are all -inf, and times the products, which are 0 too, gives the softmax's 0 / 0.
__device__ __forceinline__ float inverse(float total) { return 1.0f / total; }

// Running maximum, sum of weights and four weighted value sums.
struct Sums {
  float top, total;
  float4 x;
  __device__ __forceinline__ void add(float m, float l, const float4& y) {
    if (m == -INFINITY) {             // a part without a score above -inf: its sum of weights is 0, or NaN where a score is
      total += l;
      return;
    }
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

// A row's sums over its group's shared prefix: the (token, head of the group) row r of a sequence whose place there is `at`.
struct PreRow {
  const float* slot;
  int row;
  __device__ __forceinline__ PreRow(const SeqView& v, int2 at, int kvh, int r) {
    const int tok = at.y + r / v.G, tile = tok / v.tile_tokens;
    slot = v.pre_part + ((static_cast<int64_t>(at.x + (tile >> 1)) * v.Hkv + kvh) * 2 + (tile & 1)) * tile_slot(v);
    row = (tok - tile * v.tile_tokens) * v.G + r % v.G;
  }
  __device__ __forceinline__ float top(int hd) const { return slot[128 * hd + row]; }
  __device__ __forceinline__ float total(int hd) const { return slot[128 * hd + 128 + row]; }
  __device__ __forceinline__ float4 quad(int q) const { return reinterpret_cast<const float4*>(slot)[q * 128 + row]; }
};

// Joins `count` parts of a row kernel's item of `rows` rows (token, head of the group): those from part `from` on, `step` apart,
// of the item whose first part CTA `cta` has. The result goes to the output rows from o on (pre: with the rows' sums over their
// prefix, at pre_at in head kvh), or, without o, to the place of part `from`. All threads of the block; sx, sm: a place for each.
template <int HD, int THREADS>
__device__ __forceinline__ void join_rows(uint16_t* o, const SeqView& v, int rows, int cta, int from, int step, int count,
                                          float4* sx, float2* sm, bool pre = false, int2 pre_at = make_int2(0, 0), int kvh = 0) {
  constexpr int kQuads = HD / 4;         // groups of four columns
  const int elements = rows * kQuads;
  const int64_t slot = row_slot(v);
  float* base = v.row_part + 2 * static_cast<int64_t>(cta) * slot;            // part k > 0: base + 2 k slot
  auto part = [&](int i) {
    const int k = from + i * step;
    return base + (k == 0 ? slot : 2 * k * slot);
  };
  // threads beyond the elements take a share of the parts
  const int groups = max(1, THREADS / elements);
  float2* done = sm + THREADS;           // m and l of the rows
  for (int i0 = 0; i0 < elements; i0 += THREADS) {
    const int e = groups > 1 ? static_cast<int>(threadIdx.x) % elements : i0 + static_cast<int>(threadIdx.x);
    const int g = groups > 1 ? static_cast<int>(threadIdx.x) / elements : 0;
    const bool mine = e < elements && g < groups;
    const int r = mine ? e / kQuads : 0, h = e % kQuads * 4;
    Sums z{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (mine) {
      for (int k0 = g; k0 < count; k0 += kPartsAhead * groups) {
        float2 ml[kPartsAhead];
        float4 y[kPartsAhead];
#pragma unroll
        for (int k = 0; k < kPartsAhead; ++k) {
          const float* p = part(min(k0 + k * groups, count - 1));
          ml[k] = __ldcg(reinterpret_cast<const float2*>(p + v.row_limit * HD + 2 * r));
          y[k] = __ldcg(reinterpret_cast<const float4*>(p + r * HD + h));
        }
#pragma unroll
        for (int k = 0; k < kPartsAhead; ++k)
          if (k0 + k * groups < count) z.add(ml[k].x, ml[k].y, y[k]);
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
    if (!mine || g > 0) continue;
    if (o == nullptr) {
      *reinterpret_cast<float4*>(part(0) + r * HD + h) = z.x;                  // (no other thread reads this element)
      if (h == 0) done[r] = make_float2(z.top, z.total);
    } else {
      if (pre) {
        const PreRow p(v, pre_at, kvh, r);
        z.add(p.top(HD), p.total(HD), p.quad(h / 4));
      }
      const float inv = inverse(z.total);
      *reinterpret_cast<uint2*>(o + (static_cast<int64_t>(r / v.G) * v.Hq + r % v.G) * HD + h) =
          make_uint2(pack_bf16(z.x.x * inv, z.x.y * inv), pack_bf16(z.x.z * inv, z.x.w * inv));
    }
  }
  if (o == nullptr) {
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < rows)
      *reinterpret_cast<float2*>(part(0) + v.row_limit * HD + 2 * threadIdx.x) = done[threadIdx.x];
    __syncthreads();
  }
}

}  // namespace mlora
