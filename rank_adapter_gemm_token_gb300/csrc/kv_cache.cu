// The paged cache's own kernels.
//
// qkv_write: a step's qkv rows (the qkv linear's fp32 output) on their way to the attention. For each
// token and head of hd elements x:
//     x <- x / sqrt(mean(x^2) + eps) * w                        queries and keys, where a weight is given
//     (a, b) <- m (a cos - b sin, b cos + a sin)                 queries and keys, the first rot elements
//     queries: bf16 row of q; keys and values: row pos % page of page table[pos / page], as bf16 or as
//     e4m3 codes rn(x / s) with s = max(max |x|, 2^-60) / 448, one fp32 s for each token and head.
// A row with an infinity or a NaN gets codes 0 and the scale NaN, so that all of it reads back as NaN.
// Angles are taken in turns: pos * f with f a sum of three floats, the whole turns of each product and of its
// rounding error (by fma) dropped exactly, then sin and cos of the fraction: 2e-7 for every position up to 2^24 and
// frequency up to 1 (5e-7 up to 1e6), where an fp32 angle in radians would be off by pos * 6e-8.
// Bound: HBM, each value read once and written once, and close behind it the instructions: a row (one head of one token)
// lies in the registers of hd / 8 lanes, eight elements each, so that norm, rotation and maximum are a few shuffles for two
// (four) rows at a time, and the angles of a CTA's few tokens are made once, in shared memory. Each thread has two rows on
// their way before it works on the first, five CTAs an SM: with three rows and three CTAs fewer loads were on their way
// beside the arithmetic (40 us against 34 for 4096 tokens of 48 heads of 128, e4m3). One row for a small step. Measured on the GPU: those
// 4096 tokens 31 us, 4.6 TB/s, instructions issued in 0.76 of the cycles (bf16 with norms 35 us, 4.3 TB/s); 256 tokens 6 us. The
// two-step forms spill 68 bytes at 48 registers.
//
// kv_read: whole sequences' cached rows as dense bf16 rows [token, head, hd]; a copy (bf16) or code * scale
// rounded once (e4m3). Bound: HBM. A warp takes a run of consecutive (page, head) units, so that only its first one
// searches for its sequence. e4m3: a lane's 16 codes are 32 bytes of output, written in one store: in two, each with half
// of every sector, 64000 tokens of 8 heads took 81 us in place of 67 (5.6 TB/s of codes, scales and rows together).
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

constexpr int kPairs = 64;               // most pairs of a rotation

// A CTA: rows (token, head) from blockIdx.x * kRows on (heads: the query heads, the key heads, the value heads), a row to
// HD / 8 lanes of eight elements each, STEPS rows to each of them.
template <int HD, int STEPS>
__global__ void __launch_bounds__(kWriteWarps * 32, STEPS == 1 ? 6 : 5)
qkv_write_kernel(const float* __restrict__ qkv, int64_t ld, const uint16_t* __restrict__ q_norm,
                 const uint16_t* __restrict__ k_norm, float eps, RopeView rope, const int32_t* __restrict__ positions,
                 uint16_t* __restrict__ q, KvView kv, SeqView s) {
  constexpr int kLanes = HD / 8, kStep = kWriteWarps * 32 / kLanes, kRows = kStep * STEPS;
  constexpr int kTokens = kRows / 3 + 2;                   // of a CTA: a token has at least three rows
  __shared__ alignas(16) float2 angle[kTokens][kPairs];    // m cos, m sin
  __shared__ int cache_row[kTokens], in_seq[kTokens];
  const int heads = s.Hq + 2 * s.Hkv;
  const int64_t rows = static_cast<int64_t>(s.T) * heads, row0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int t0 = static_cast<int>(row0 / heads), h0 = static_cast<int>(row0 - static_cast<int64_t>(t0) * heads);
  const int tokens = min((h0 + kRows - 1) / heads + 1, s.T - t0), half = rope.rot >> 1;
  if (threadIdx.x < tokens) {
    cache_row[threadIdx.x] = s.tok_row[t0 + threadIdx.x];
    in_seq[threadIdx.x] = s.tok_seq[t0 + threadIdx.x] >= 0;
  }
  // this thread's first angle (with few tokens the only one): its position is on its way before the rows are
  int at = 0, ak = threadIdx.x;
  if (half > 0 && ak >= half) at = ak / half, ak -= at * half;
  float pos = 0.f;
  if (half > 0 && at < tokens) pos = static_cast<float>(positions ? positions[t0 + at] : s.tok_pos[t0 + at]);

  // The lane's two quads of elements: neighbours, or, for whole heads in the half layout, the two quads of the same pairs
  const int lane = threadIdx.x & 31, le = threadIdx.x % kLanes;
  const bool split = !rope.interleaved && rope.rot == HD;
  const int e0 = split ? 4 * le : 8 * le, e1 = split ? e0 + HD / 2 : e0 + 4;
  float x[STEPS][8];
  int tl[STEPS], head[STEPS];            // token (from t0) and head of each row (-1: none)
  {
    const int left = static_cast<int>(min(rows - row0, static_cast<int64_t>(kRows)));
    const float* src = qkv + t0 * ld;
    int t = 0, h = h0 + threadIdx.x / kLanes;
    if (h >= heads) t = h / heads, h -= t * heads;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const bool mine = static_cast<int>(threadIdx.x) / kLanes + i * kStep < left;
      tl[i] = mine ? t : 0, head[i] = mine ? h : -1;
      const float* p = src + t * ld + h * HD;
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 a = mine ? __ldcs(reinterpret_cast<const float4*>(p + e0)) : zero;
      const float4 b = mine ? __ldcs(reinterpret_cast<const float4*>(p + e1)) : zero;
      x[i][0] = a.x, x[i][1] = a.y, x[i][2] = a.z, x[i][3] = a.w;
      x[i][4] = b.x, x[i][5] = b.y, x[i][6] = b.z, x[i][7] = b.w;
      h += kStep;
      while (h >= heads) h -= heads, ++t;
    }
  }
  if (half > 0) {
    while (at < tokens) {
      const float4 f = __ldg(rope.freq + ak);
      const float p = pos * f.x, p1 = pos * f.y, r = fmaf(pos, f.x, -p);
      float frac = p - rintf(p);
      frac += (r - rintf(r)) + (p1 - rintf(p1)) + (fmaf(pos, f.y, -p1) + pos * f.z);
      float sn, cs;
      sincospif(2.0f * frac, &sn, &cs);
      angle[at][ak] = make_float2(cs * rope.mscale, sn * rope.mscale);
      ak += kWriteWarps * 32;
      at += ak / half;
      ak %= half;
      if (at < tokens) pos = static_cast<float>(positions ? positions[t0 + at] : s.tok_pos[t0 + at]);
    }
  }
  // The quads' pairs' angles, and where the pairs' other elements are (half layout: quads n further or nearer; n odd: in the
  // other place of their lane).
  const int n = half >> 2;
  const bool odd = !rope.interleaved && (n & 1);
  bool turned[2];
  int first_pair[2], from[2];
  float sign[2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int quad = (b ? e1 : e0) >> 2;
    turned[b] = quad * 4 < rope.rot;
    const bool second = quad >= n;
    first_pair[b] = !turned[b] ? 0 : rope.interleaved ? 2 * quad : 4 * (second ? quad - n : quad);
    from[b] = (lane & ~(kLanes - 1)) + ((!turned[b] ? quad : second ? quad - n : quad + n) >> 1);
    sign[b] = second ? 1.f : -1.f;
  }
  uint4 qn = make_uint4(0u, 0u, 0u, 0u), kn = qn;
  auto weights = [&](const uint16_t* w) {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(w + e0)), b = __ldg(reinterpret_cast<const uint2*>(w + e1));
    return make_uint4(a.x, a.y, b.x, b.y);
  };
  if (q_norm) qn = weights(q_norm);
  if (k_norm) kn = weights(k_norm);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int h = head[i];
    const bool is_q = h >= 0 && h < s.Hq, is_k = h >= s.Hq && h < s.Hq + s.Hkv;
    if ((q_norm || k_norm) && __any_sync(0xffffffffu, is_q || is_k)) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(x[i][j], x[i][j], sum);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if ((is_q && q_norm) || (is_k && k_norm)) {
        const float r = rsqrtf(sum * (1.0f / HD) + eps);
        const uint4 w = is_q ? qn : kn;
        const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][2 * j] *= r * ptx::bf16_lo(y[j]);
          x[i][2 * j + 1] *= r * ptx::bf16_hi(y[j]);
        }
      }
    }
    if (half > 0 && __any_sync(0xffffffffu, is_q || is_k)) {
      float other[8];
      if (split) {
#pragma unroll
        for (int j = 0; j < 8; ++j) other[j] = x[i][j ^ 4];
      } else if (!rope.interleaved) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) other[4 * b + j] = __shfl_sync(0xffffffffu, odd ? x[i][4 * (b ^ 1) + j] : x[i][4 * b + j], from[b]);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (!turned[b] || !(is_q || is_k)) continue;
        const float4* a = reinterpret_cast<const float4*>(&angle[tl[i]][first_pair[b]]);
        float* y = &x[i][4 * b];
        const float4 t = a[0];
        if (rope.interleaved) {
          const float u0 = y[0], u1 = y[2];
          y[0] = u0 * t.x - y[1] * t.y;
          y[1] = y[1] * t.x + u0 * t.y;
          y[2] = u1 * t.z - y[3] * t.w;
          y[3] = y[3] * t.z + u1 * t.w;
        } else {
          const float4 t1 = a[1];
          const float* z = &other[4 * b];
          y[0] = y[0] * t.x + z[0] * (t.y * sign[b]);
          y[1] = y[1] * t.z + z[1] * (t.w * sign[b]);
          y[2] = y[2] * t1.x + z[2] * (t1.y * sign[b]);
          y[3] = y[3] * t1.z + z[3] * (t1.w * sign[b]);
        }
      }
    }
    uint4 bf;
    bf.x = pack_bf16(x[i][0], x[i][1]);
    bf.y = pack_bf16(x[i][2], x[i][3]);
    bf.z = pack_bf16(x[i][4], x[i][5]);
    bf.w = pack_bf16(x[i][6], x[i][7]);
    const int row = cache_row[tl[i]];
    uint32_t most = 0;                   // (magnitudes order as their bit patterns do, infinities and NaN above all)
    if (kv.type == kKvE4m3 && __any_sync(0xffffffffu, h >= s.Hq)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) most = max(most, __float_as_uint(x[i][j]) & 0x7fffffffu);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    }
    if (is_q) {
      if (!in_seq[tl[i]]) bf = make_uint4(0u, 0u, 0u, 0u);
      uint16_t* dst = q + (static_cast<int64_t>(t0 + tl[i]) * s.Hq + h) * HD;
      *reinterpret_cast<uint2*>(dst + e0) = make_uint2(bf.x, bf.y);
      *reinterpret_cast<uint2*>(dst + e1) = make_uint2(bf.z, bf.w);
    } else if (h >= 0 && row >= 0) {
      const int kh = is_k ? h - s.Hq : h - s.Hq - s.Hkv;
      const int64_t to = ((static_cast<int64_t>(row >> kv.page_log2) * kv.Hkv + kh) << kv.page_log2) + (row & (kv.page - 1));
      void* base = is_k ? kv.K : kv.V;
      if (kv.type == kKvBf16) {
        uint16_t* dst = static_cast<uint16_t*>(base) + to * HD;
        *reinterpret_cast<uint2*>(dst + e0) = make_uint2(bf.x, bf.y);
        *reinterpret_cast<uint2*>(dst + e1) = make_uint2(bf.z, bf.w);
      } else {
        const bool finite = most < 0x7f800000u;
        const float scale = finite ? fmaxf(__uint_as_float(most), kAmaxMin) * (1.0f / kE4m3Max) : __int_as_float(0x7fffffff);
        const float inv = __fdividef(1.0f, scale);
        uint2 c = make_uint2(0u, 0u);
        if (finite) {
          c.x = pack_e4m3(x[i][0] * inv, x[i][1] * inv) | (pack_e4m3(x[i][2] * inv, x[i][3] * inv) << 16);
          c.y = pack_e4m3(x[i][4] * inv, x[i][5] * inv) | (pack_e4m3(x[i][6] * inv, x[i][7] * inv) << 16);
        }
        uint8_t* dst = static_cast<uint8_t*>(base) + to * HD;
        *reinterpret_cast<uint32_t*>(dst + e0) = c.x;
        *reinterpret_cast<uint32_t*>(dst + e1) = c.y;
        if (le == 0) (is_k ? kv.k_scale : kv.v_scale)[to] = scale;
      }
    }
  }
}

constexpr int kReadWarps = 8;
constexpr int kReadCtas = 4;             // of an SM

// A warp: a run of (page, head) units of the step's cached pages, K and V; 16 bytes of cached row a lane.
template <int HD, bool E4M3>
__global__ void __launch_bounds__(kReadWarps * 32, kReadCtas)
kv_read_kernel(const int32_t* __restrict__ row_start, int64_t rows, uint16_t* __restrict__ k_out,
               uint16_t* __restrict__ v_out, KvView kv, SeqView s) {
  constexpr int kE = E4M3 ? 16 : 8;                       // elements of a lane
  constexpr int kLanes = HD / kE, kStep = 32 / kLanes;    // lanes of a row, rows of a step
  constexpr int kAhead = E4M3 ? 2 : 4;                    // steps asked for at once
  const int lane = threadIdx.x & 31;
  const int64_t units = static_cast<int64_t>(s.page_pre[s.S]) * kv.Hkv;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5), warps = static_cast<int64_t>(gridDim.x) * kReadWarps;
  int64_t u = units * w / warps;
  const int64_t end = units * (w + 1) / warps;
  if (u >= end) return;
  const int e = lane % kLanes * kE, r0 = lane / kLanes;
  const bool wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31) == 0;
  int g = static_cast<int>(u / kv.Hkv), h = static_cast<int>(u - static_cast<int64_t>(g) * kv.Hkv);
  int sq = last_at_most(s.page_pre, s.S, g);
  while (u < end) {
    const int first = s.page_pre[sq], next = s.page_pre[sq + 1], len = s.len[sq];
    const int64_t start = row_start[sq];
    for (; g < next && u < end; ++g, h = 0) {             // the sequence's pages
      const int pi = g - first, cnt = min(kv.page, len - (pi << kv.page_log2));
      const int64_t dst = start + (static_cast<int64_t>(pi) << kv.page_log2);
      const int64_t page = s.table[static_cast<size_t>(sq) * s.max_pages + pi];
      const bool fits = dst >= 0 && dst + cnt <= rows;
      if (!fits && lane == 0) atomicOr(s.err, ptx::kErrBadRow);
      for (; h < kv.Hkv && u < end; ++h, ++u) {
        if (!fits || page < 0) continue;                  // (a page that has gone out of every window)
        const int64_t at = (page * kv.Hkv + h) << kv.page_log2;
        for (int b = r0; b < cnt; b += kStep * kAhead) {
          uint4 a[kAhead], c[kAhead];
          float ks[kAhead], vs[kAhead];
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int r = min(b + k * kStep, cnt - 1);
            const int64_t from = (at + r) * HD + e;
            a[k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv.K) + from * (E4M3 ? 1 : 2)));
            c[k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv.V) + from * (E4M3 ? 1 : 2)));
            if (E4M3) ks[k] = kv.k_scale[at + r], vs[k] = kv.v_scale[at + r];
          }
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int r = b + k * kStep;
            if (r >= cnt) break;
            const int64_t to = ((dst + r) * kv.Hkv + h) * HD + e;
            if (E4M3) {
              uint4 y[2] = {e4m3_times(make_uint2(a[k].x, a[k].y), ks[k]), e4m3_times(make_uint2(a[k].z, a[k].w), ks[k])};
              store32(k_out + to, &y[0].x, wide);
              y[0] = e4m3_times(make_uint2(c[k].x, c[k].y), vs[k]), y[1] = e4m3_times(make_uint2(c[k].z, c[k].w), vs[k]);
              store32(v_out + to, &y[0].x, wide);
            } else {
              *reinterpret_cast<uint4*>(k_out + to) = a[k];
              *reinterpret_cast<uint4*>(v_out + to) = c[k];
            }
          }
        }
      }
      if (h < kv.Hkv) return;                             // the run ends inside the page
    }
    while (sq < s.S && s.page_pre[sq + 1] <= g) ++sq;     // the next sequence with pages
  }
}

template <int HD, int STEPS>
cudaError_t write_as(const float* qkv, int64_t ld, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                     const RopeView& rope, const int32_t* positions, uint16_t* q, const KvView& kv, const SeqView& s,
                     cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(s.T) * (s.Hq + 2 * s.Hkv);
  constexpr int kRows = kWriteWarps * 32 * 8 / HD * STEPS;
  const int grid = static_cast<int>((rows + kRows - 1) / kRows);
  note_launch_begin(kKindKv, st);
  qkv_write_kernel<HD, STEPS><<<grid, kWriteWarps * 32, 0, st>>>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s);
  const cudaError_t e = cudaGetLastError();
  note_launch_end(kKindKv, st);
  return e;
}

}  // namespace

cudaError_t launch_qkv_write(const float* qkv, int64_t ld, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                             const RopeView& rope, const int32_t* positions, uint16_t* q, const KvView& kv,
                             const SeqView& s, int num_sms, cudaStream_t st) {
  if (s.T == 0) return cudaSuccess;
  // One step while two would leave SMs without work: shorter for the few tokens of a small step.
  const bool few = static_cast<int64_t>(s.T) * (s.Hq + 2 * s.Hkv) * s.hd < 4096L * num_sms;
  if (s.hd == 128)
    return few ? write_as<128, 1>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st)
               : write_as<128, 2>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st);
  return few ? write_as<64, 1>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st)
             : write_as<64, 2>(qkv, ld, q_norm, k_norm, eps, rope, positions, q, kv, s, st);
}

cudaError_t launch_kv_read(const int32_t* row_start, int64_t rows, uint16_t* k, uint16_t* v, const KvView& kv,
                           const SeqView& s, int num_sms, cudaStream_t st) {
  if (s.S == 0) return cudaSuccess;
  const int64_t most = std::max<int64_t>(1, (rows / kv.page + s.S) * kv.Hkv);      // units of a call that fits
  const int grid = static_cast<int>(std::min<int64_t>((most + kReadWarps - 1) / kReadWarps, static_cast<int64_t>(kReadCtas) * num_sms));
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
