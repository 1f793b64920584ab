// Attention of sequences with few query rows (single tokens, short chunks) over the paged cache:
//
//     o_r = sum_{j <= p_r} softmax_j(scale q_r . k_j) v_j
//
// for the rows r = (token i, head of the group) of one key/value head, p_r the token's position.
// Bound: HBM. Each cached row is read once and meets at most 16 query rows (2 to 4 flops a byte), so the
// work is to keep loads in flight and the split even:
//   - work = (sequence, key/value head) items of 64-key units, laid out one after another; every CTA takes an
//     equal share of the units whatever the sequences' lengths (Shares), so one long sequence and many short
//     ones both fill the GPU. An item across a cut leaves partial sums (with their maximum) in the step's
//     workspace, and the CTA that comes last with one joins them in their order: the result does not depend on who it is.
//     (As a launch of its own that took as long on the GPU, and a small call 2 us more.)
//   - a warp takes 16 keys of each unit, through its own ring of stages filled by cp.async (the next item's
//     keys are already on their way while one item is finished), with no barrier between warps inside an item.
//   - the products run on the warp-level tensor instructions with the keys as the M side: S^T = K Q^T and
//     O^T = V^T P^T with the query rows as N = 8 (or 16), so few rows waste few lanes. (The tcgen05 shapes need
//     128 rows; here the tensor time is a fraction of the load time either way.)
//   - softmax in one pass in base 2; the running maximum moves only when a score passes it by 2^8, so most
//     chunks need no shuffles and no rescaling. bf16: P meets the values in two pieces of 8 bits, which costs a second
//     product where the tensor cores wait for loads anyway (256 sequences 168.5 us without it, 169.8 with). e4m3: one piece, f16's 11
//     bits (a second would cost 4 %: 105.8 us, 109.9).
//   - e4m3: codes become f16 (exact) in registers. The key scale multiplies the score. The weights w_j = 2^(score_j - m)
//     go into the denominator as they are; for the product with the codes they are multiplied by the value scale and by
//     u = 2^(m - n), where n + 7 follows the largest score_j + log2 vs_j as m follows the largest score: P_j = w_j vs_j u is at
//     most 2^15 whatever the scales' magnitude. A value scale of 0 leaves its weight in the denominator. Both maxima
//     are whole numbers, so every rescaling is exact. Query rows are lifted by a power of two into f16's range.
// Keys at or past a row's limit are replaced by -inf by selection, and rows past the cached length are
// zero-filled on load, so what lies there (NaN included) has no effect.
// Measured on the GPU, 32 heads of 128 on 8, all bytes over the time: 256 sequences of 200-2000 tokens bf16 168 us, 6.6 TB/s;
// e4m3 105 us, 5.8 TB/s; one of 131000 tokens 84 us, 6.4 TB/s (copy: 6.8), e4m3 51 us, 5.4; one of 500 tokens 7.5 us. 9 to 16 rows
// (64 sequences of 3 tokens on 1000): 54 us, 4.9 TB/s; e4m3 46 us, 3.0.
#include <algorithm>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 16;                  // keys of a warp's chunk
constexpr float kLazy = 8.0f;               // log2 of the largest weight; e4m3: of the largest weight times scale, before
constexpr float kUp = 7.0f;                 // P is lifted to the top of f16's range: its normal numbers then reach down to 2^-21
constexpr float kMostP = 32768.0f;          // of the row's largest
// A value scale counts as this power of two at least where the maximum is taken: the maximum of value rows of scale 0 alone
// stays finite, and 2^80 times any number of weights does too.
constexpr float kLeastLog2 = -80.0f;

template <int HD, int NQ, bool E4M3>
struct RowsCfg {
  static constexpr int kRowBytes = E4M3 ? HD : 2 * HD;
  static constexpr int kSegs = kRowBytes / 16;                     // 16-byte segments of a cached row
  static constexpr int kTile = kChunk * kRowBytes;
  static constexpr int kScales = E4M3 ? 2 * kChunk * 4 : 0;        // key and value scales of a chunk
  static constexpr int kStage = 2 * kTile + kScales;
  // CTAs of an SM, and bytes of a CTA's stages: e4m3 chunks are half as long and take more instructions, so they get
  // more warps.
  static constexpr int kCtas = rows_ctas_per_sm(NQ == 2, E4M3);
  static constexpr int kRing = kCtas == 3 ? 54 * 1024 : NQ == 1 ? 96 * 1024 : 64 * 1024;
  static constexpr int kStages = kRing / (kWarps * kStage) > 8 ? 8 : kRing / (kWarps * kStage);
  static constexpr int kRows = 8 * NQ;
  static constexpr int kLd = HD + 4;                               // floats of a row of the joined sums
  static constexpr int kOOff = kWarps * kStages * kStage;
  static constexpr int kMlOff = kOOff + kWarps * kRows * kLd * 4;
  static constexpr int kBytes = kMlOff + kWarps * kRows * 2 * 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(full ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t mat_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A power of two from its exponent (a whole number in [-126, 127]), and back.
__device__ __forceinline__ float pow2_of(float x) { return __int_as_float((static_cast<int>(x) + 127) << 23); }
__device__ __forceinline__ float log2_of(float x) { return static_cast<float>((__float_as_int(x) >> 23) - 127); }

// A place in the list of units: unit u of head kvh of list entry i.
struct Place {
  int i, kvh, u, units;
  RowSeq s;
  const int32_t* table;
  __device__ __forceinline__ void load(const SeqView& v) {
    const int4 x = *reinterpret_cast<const int4*>(v.row_seq + i);
    s = RowSeq{x.x, x.y, x.z, x.w};
    units = (s.len + kRowUnit - 1) / kRowUnit;
    table = v.table + static_cast<size_t>(s.seq) * v.max_pages;
  }
  // the next unit; the caller knows that there is one
  __device__ __forceinline__ void next(const SeqView& v) {
    if (++u < units) return;
    u = 0;
    if (++kvh < v.Hkv) return;
    kvh = 0;
    ++i;
    load(v);
  }
};

template <int HD, int NQ, bool E4M3>
__global__ void __launch_bounds__(kThreads, RowsCfg<HD, NQ, E4M3>::kCtas)
attention_rows_kernel(const uint16_t* __restrict__ q, uint16_t* __restrict__ o, float scale_log2, KvView kv, SeqView v) {
  using C = RowsCfg<HD, NQ, E4M3>;
  constexpr int kSteps = HD / 16;             // k-steps of S^T, M tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  float* o_sh = reinterpret_cast<float*>(smem + C::kOOff);
  float* ml_sh = reinterpret_cast<float*>(smem + C::kMlOff);
  ptx::grid_dependents_launch();

  const int4 share = *reinterpret_cast<const int4*>(v.row_share + blockIdx.x);
  const int n_chunks = share.w;
  // ---- the warp's loads: chunk i of the CTA's share goes to stage i % kStages
  const uint32_t ring = ptx::smem_u32(smem) + warp * (C::kStages * C::kStage);
  Place src{share.x, share.y, share.z, 0, {}, nullptr};
  int issued = 0;
  int page_a = 0, page_b = 0;                 // pages of the next chunk's first and second 8 keys
  auto look = [&]() {
    const int k0 = src.u * kRowUnit + warp * kChunk;
    page_a = src.table[min(k0, src.s.len - 1) >> kv.page_log2];
    page_b = kv.page_log2 < 4 ? src.table[min(k0 + 8, src.s.len - 1) >> kv.page_log2] : page_a;
  };
  if (n_chunks > 0) {
    src.load(v);
    look();
  }
  auto issue = [&]() {
    if (issued < n_chunks) {
      const int k0 = src.u * kRowUnit + warp * kChunk;
      if (k0 < src.s.len) {
        const uint32_t st = ring + (issued % C::kStages) * C::kStage;
        constexpr int kStep = 32 / C::kSegs;  // rows of one copy of all lanes
        constexpr int kHalf = kChunk / 2 / kStep;                                // copies of eight rows
        static_assert(kStep * kHalf == 8, "a copy of all lanes takes 2, 4 or 8 rows");
        // the chunk's first and second eight rows: pages of 16 tokens and more hold them one after the other
        const int64_t row_a = (static_cast<int64_t>(page_a) * v.Hkv + src.kvh) << kv.page_log2;
        const int64_t row_b = (static_cast<int64_t>(page_b) * v.Hkv + src.kvh) << kv.page_log2;
        const int off_a = k0 & (kv.page - 1), off_b = (k0 + 8) & (kv.page - 1);
        const int lr = lane / C::kSegs, seg = lane % C::kSegs;
        const bool full = k0 + kChunk <= src.s.len;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int64_t at = ((half ? row_b + off_b : row_a + off_a) + lr) * C::kRowBytes + seg * 16;
          const uint8_t* pk = static_cast<const uint8_t*>(kv.K) + at;
          const uint8_t* pv = static_cast<const uint8_t*>(kv.V) + at;
#pragma unroll
          for (int i = 0; i < kHalf; ++i) {
            const int r = half * 8 + i * kStep + lr;
            const int phys = C::kSegs >= 8 ? seg ^ (r & 7) : seg ^ ((r >> 1) & 3);
            const uint32_t dst = st + r * C::kRowBytes + phys * 16;
            const bool in = full || k0 + r < src.s.len;
            cp16(dst, pk + i * kStep * C::kRowBytes, in);
            cp16(dst + C::kTile, pv + i * kStep * C::kRowBytes, in);
          }
        }
        if (E4M3) {
          const int r = lane & 15;
          const int64_t at = (r < 8 ? row_a + off_a : row_b + off_b) + (r & 7);
          cp4(st + 2 * C::kTile + lane * 4, (lane < 16 ? kv.k_scale : kv.v_scale) + at, full || k0 + r < src.s.len);
        }
      }
      ++issued;
      if (issued < n_chunks) {
        src.next(v);
        look();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) issue();

  // rows of tokens in no sequence are zero
  for (int t0 = blockIdx.x * 32; t0 < v.T; t0 += gridDim.x * 32) {
    const int tok = t0 + lane;
    uint32_t none = __ballot_sync(0xffffffffu, tok < v.T && v.tok_seq[tok] < 0);
    none &= 0x11111111u << warp;
    while (none) {
      const int b = __ffs(none) - 1;
      none &= none - 1;
      uint4* row = reinterpret_cast<uint4*>(o + static_cast<int64_t>(t0 + b) * v.Hq * HD);
      for (int i = lane; i < v.Hq * HD / 8; i += 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // ---- the CTA's items
  Place at{share.x, share.y, share.z, 0, {}, nullptr};
  if (n_chunks > 0) at.load(v);
  int done = 0;
  while (done < n_chunks) {
    const int u_end = min(at.units, at.u + (n_chunks - done));
    const int n = at.s.n, first = at.s.start, len = at.s.len;
    const int rows = n * v.G;
    const int base = len - n;                  // position of the first new token
    uint32_t bq[NQ][kSteps][2];
    float cq[NQ][2];
    int lim[NQ][2];
#pragma unroll
    for (int z = 0; z < NQ; ++z) {
      const int r = z * 8 + g;
      const uint16_t* row = q + (static_cast<int64_t>(first + (r < rows ? r / v.G : 0)) * v.Hq + at.kvh * v.G + (r < rows ? r % v.G : 0)) * HD;
      if (E4M3) {
        uint4 w[kSteps / 2];
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i) {
          w[i] = r < rows ? *reinterpret_cast<const uint4*>(row + t * (HD / 4) + i * 8) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t* p = &w[i].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) most = fmaxf(most, fmaxf(fabsf(ptx::bf16_lo(p[k])), fabsf(ptx::bf16_hi(p[k]))));
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        float back;
        const float lift = query_lift(most, &back);
#pragma unroll
        for (int i = 0; i < kSteps / 2; ++i) {
          const uint32_t* p = &w[i].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) bq[z][2 * i + (k >> 1)][k & 1] = pack_f16(ptx::bf16_lo(p[k]) * lift, ptx::bf16_hi(p[k]) * lift);
        }
        cq[z][0] = scale_log2 * __shfl_sync(0xffffffffu, back, (2 * t) * 4);
        cq[z][1] = scale_log2 * __shfl_sync(0xffffffffu, back, (2 * t + 1) * 4);
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          bq[z][i][0] = r < rows ? *reinterpret_cast<const uint32_t*>(row + 16 * i + 2 * t) : 0u;
          bq[z][i][1] = r < rows ? *reinterpret_cast<const uint32_t*>(row + 16 * i + 2 * t + 8) : 0u;
        }
        cq[z][0] = cq[z][1] = scale_log2;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int rc = z * 8 + 2 * t + c;
        lim[z][c] = rc < rows ? base + rc / v.G : -1;
      }
    }
    float acc[NQ][kSteps][4], m[NQ][2], l[NQ][2];
    float up[NQ][2];                           // e4m3: 2^(m - n), a power of two
#pragma unroll
    for (int z = 0; z < NQ; ++z) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[z][i][k] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) m[z][c] = -INFINITY, l[z][c] = 0.f, up[z][c] = 1.f;
    }

    for (int u = at.u; u < u_end; ++u, ++done) {
      cp_wait<C::kStages - 2>();
      __syncwarp();
      issue();
      const int k0 = u * kRowUnit + warp * kChunk;
      if (k0 >= len) continue;
      const uint32_t st = ring + (done % C::kStages) * C::kStage;
      float ks[2] = {1.f, 1.f}, vs[2] = {1.f, 1.f};
      if (E4M3) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ks[h] = lds_f(st + 2 * C::kTile + (g + 8 * h) * 4);
          vs[h] = lds_f(st + 2 * C::kTile + 64 + (g + 8 * h) * 4);
          if (vs[h] < kLeastScale) vs[h] = 0.f;
        }
      }
      float sc[NQ][4], sc1[NQ][4];                // two sums, of the even and odd k-steps: half the chain of products
#pragma unroll
      for (int z = 0; z < NQ; ++z)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[z][k] = sc1[z][k] = 0.f;
      if (E4M3) {
        // lane (g, t): bytes t HD/4 ... of key rows g and g + 8; byte 4 i + j is k index (2 t + (j & 1) + 8 (j >> 1))
        // of step i, for the query rows alike
        uint4 w[2][HD / 64];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < HD / 64; ++i) {
            const int r = g + 8 * h, seg = t * (HD / 64) + i;
            w[h][i] = lds16(st + r * C::kRowBytes + (C::kSegs >= 8 ? seg ^ (r & 7) : seg ^ ((r >> 1) & 3)) * 16);
          }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const uint32_t x = (&w[0][i >> 2].x)[i & 3], y = (&w[1][i >> 2].x)[i & 3];
          uint32_t a[4];
          e4m3x4_f16x4(x, a[0], a[2]);
          e4m3x4_f16x4(y, a[1], a[3]);
#pragma unroll
          for (int z = 0; z < NQ; ++z) mma<true>(i & 1 ? sc1[z] : sc[z], a, bq[z][i][0], bq[z][i][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint32_t a[4];
          const int r = lane & 15, seg = 2 * i + (lane >> 4);
          ldsm4(a, st + r * C::kRowBytes + (seg ^ (r & 7)) * 16);
#pragma unroll
          for (int z = 0; z < NQ; ++z) mma<false>(i & 1 ? sc1[z] : sc[z], a, bq[z][i][0], bq[z][i][1]);
        }
      }
      uint32_t pb[NQ][2], pr[NQ][2];              // P in 16 bits, and (bf16) what that leaves, in 16 more
      const bool edge = k0 + kChunk > base + 1;
#pragma unroll
      for (int z = 0; z < NQ; ++z) {
        bool grow = false;
        uint32_t hidden = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = k & 1, h = k >> 1;
          float x = sc[z][k] + sc1[z][k];
          x = E4M3 ? x * ks[h] * cq[z][c] : x * cq[z][c];
          if (edge && k0 + g + 8 * h > lim[z][c]) x = -INFINITY, hidden |= 1u << k;
          sc[z][k] = x;
          grow = grow || x > m[z][c] + kLazy;
        }
        float w[4], p[4];                         // weights, and times scale and u
        auto weights = [&]() {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = k & 1, h = k >> 1;
            w[k] = exp2_approx(sc[z][k] - (m[z][c] == -INFINITY ? 0.f : m[z][c]));
            // (what a row does not see counts nothing, also where its scale is NaN)
            p[k] = !E4M3 ? w[k] : hidden >> k & 1 ? 0.f : w[k] * (vs[h] * up[z][c]);
          }
        };
        if (E4M3) {
          weights();
#pragma unroll
          for (int k = 0; k < 4; ++k) grow = grow || p[k] > kMostP;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            auto over_keys = [&](float top) {
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              return top;
            };
            float top = over_keys(fmaxf(sc[z][c], sc[z][2 + c]));
            if (E4M3) top = ceilf(top);
            top = fmaxf(top, m[z][c]);
            const float f = top == m[z][c] ? 1.f : exp2_approx(m[z][c] - top);
            float fp = f;
            if (E4M3) {
              float t[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) t[h] = sc[z][2 * h + c] + fmaxf(__log2f(vs[h]), kLeastLog2);
              const float old = m[z][c] - log2_of(up[z][c]);
              const float next = fminf(fmaxf(ceilf(over_keys(fmaxf(t[0], t[1]))) - kUp, old), top + 126.f);
              fp = next == old ? 1.f : exp2_approx(old - next);
              if (top != -INFINITY) up[z][c] = pow2_of(top - next);
            }
            m[z][c] = top;
            l[z][c] *= f;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) acc[z][i][c] *= fp, acc[z][i][2 + c] *= fp;
          }
          if (E4M3) weights();
        }
        if (!E4M3) weights();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          l[z][k & 1] += w[k];
          sc[z][k] = p[k];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = sc[z][2 * h], p1 = sc[z][2 * h + 1];
          const uint32_t x = E4M3 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
          pb[z][h] = mat_trans(x);
          if (!E4M3) pr[z][h] = mat_trans(pack_bf16(p0 - ptx::bf16_lo(x), p1 - ptx::bf16_hi(x)));
        }
      }
      const uint32_t vt = st + C::kTile;
      if (E4M3) {
        // lane (g, t): bytes g HD/8 ... of value rows 2t, 2t + 1, 2t + 8, 2t + 9; byte 2 i (+ 1) is row g (+ 8) of M tile i
        uint32_t w[4][HD / 32];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int r = 2 * t + (h & 1) + 8 * (h >> 1);
          if (HD == 128) {
            *reinterpret_cast<uint4*>(w[h]) = lds16(vt + r * C::kRowBytes + (g ^ (r & 7)) * 16);
          } else {
            *reinterpret_cast<uint2*>(w[h]) = lds8(vt + r * C::kRowBytes + ((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8);
          }
        }
#pragma unroll
        for (int j = 0; j < HD / 32; ++j) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t x = __byte_perm(w[0][j], w[1][j], b ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(w[2][j], w[3][j], b ? 0x7362 : 0x5140);
            uint32_t a[4];
            e4m3x4_f16x4(x, a[0], a[1]);
            e4m3x4_f16x4(y, a[2], a[3]);
#pragma unroll
            for (int z = 0; z < NQ; ++z) mma<true>(acc[z][2 * j + b], a, pb[z][0], pb[z][1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint32_t a[4];
          const int r = (lane & 7) + ((lane >> 4) & 1) * 8, seg = 2 * i + ((lane >> 3) & 1);
          ldsm4t(a, vt + r * C::kRowBytes + (seg ^ (r & 7)) * 16);
#pragma unroll
          for (int z = 0; z < NQ; ++z) {
            mma<false>(acc[z][i], a, pb[z][0], pb[z][1]);
            mma<false>(acc[z][i], a, pr[z][0], pr[z][1]);
          }
        }
      }
    }

    // ---- the warps' sums joined
#pragma unroll
    for (int z = 0; z < NQ; ++z)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[z][c] += __shfl_xor_sync(0xffffffffu, l[z][c], d);
        const int r = z * 8 + 2 * t + c;
        if (g == 0) {
          // (e4m3: from here on by the maximum that the value sums go by)
          ml_sh[(warp * C::kRows + r) * 2] = E4M3 ? m[z][c] - log2_of(up[z][c]) : m[z][c];
          ml_sh[(warp * C::kRows + r) * 2 + 1] = E4M3 ? l[z][c] * up[z][c] : l[z][c];
        }
        float* row = o_sh + (warp * C::kRows + r) * C::kLd;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int h0 = E4M3 ? (HD / 8) * g + 2 * i : 16 * i + g, h1 = E4M3 ? h0 + 1 : h0 + 8;
          row[h0] = acc[z][i][c];
          row[h1] = acc[z][i][2 + c];
        }
      }
    __syncthreads();
    constexpr int kGroups = HD / 8;
    auto write_out = [&](int r, int h, const float* x, float total) {
      const float inv = inverse(total);
      uint4 w;
      w.x = pack_bf16(x[0] * inv, x[1] * inv);
      w.y = pack_bf16(x[2] * inv, x[3] * inv);
      w.z = pack_bf16(x[4] * inv, x[5] * inv);
      w.w = pack_bf16(x[6] * inv, x[7] * inv);
      *reinterpret_cast<uint4*>(o + (static_cast<int64_t>(first + r / v.G) * v.Hq + at.kvh * v.G + r % v.G) * HD + h) = w;
    };
    const bool whole = at.u == 0 && u_end == at.units;
    float* slot = v.row_part + (2 * static_cast<int64_t>(blockIdx.x) + (at.u == 0 ? 1 : 0)) * row_slot(v);
    for (int i = threadIdx.x; i < rows * kGroups; i += kThreads) {
      const int r = i / kGroups, h = (i % kGroups) * 8;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml_sh[(w * C::kRows + r) * 2]);
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, total = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = ml_sh[(w * C::kRows + r) * 2];
        const float f = mw == -INFINITY ? 0.f : exp2_approx(mw - top);
        total = fmaf(f, ml_sh[(w * C::kRows + r) * 2 + 1], total);
        const float* row = o_sh + (w * C::kRows + r) * C::kLd + h;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = fmaf(f, row[k], x[k]);
      }
      if (whole) {
        write_out(r, h, x, total);
      } else {
        float4* p = reinterpret_cast<float4*>(slot + r * HD + h);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (h == 0) *reinterpret_cast<float2*>(slot + C::kRows * HD + 2 * r) = make_float2(top, total);
      }
    }
    __syncthreads();
    if (!whole) {
      // The CTA that comes last with a part joins them; of more than eight, runs of eight first, then the runs: with all
      // parts of a long axis read by one CTA, three sequences of 10000-40000 (38 parts an item, e4m3) took 40 us against 32.
      const int4 ends = reinterpret_cast<const int4*>(v.row_share + blockIdx.x)[1];
      const int cta = at.u > 0 ? ends.x : ends.z, parts = at.u > 0 ? ends.y : ends.w;
      auto is_last = [&](int32_t* there, int count) {
        if (threadIdx.x == 0) {
          __threadfence();
          const bool last = atomicAdd(there, 1) == count - 1;
          if (last) *there = 0;                       // for the next call
          __threadfence();
          ml_sh[0] = last ? 1.f : 0.f;
        }
        __syncthreads();
        const bool last = ml_sh[0] != 0.f;
        __syncthreads();
        return last;
      };
      float4* sx = reinterpret_cast<float4*>(o_sh);
      float2* sm = reinterpret_cast<float2*>(o_sh + 4 * kThreads);
      uint16_t* out = o + (static_cast<int64_t>(first) * v.Hq + at.kvh * v.G) * HD;
      const int run = (static_cast<int>(blockIdx.x) - cta) & ~(kPartsAhead - 1), in_run = min(kPartsAhead, parts - run);
      // (an item's first run and the last of the item before may begin in the same CTA: counters of their own)
      if (is_last(v.row_there + (run == 0 ? 0 : 2 * v.row_ctas) + cta + run, in_run)) {
        const bool all = parts <= kPartsAhead;
        join_rows<HD, kThreads>(all ? out : nullptr, v, rows, cta, run, 1, in_run, sx, sm);
        const int runs = (parts + kPartsAhead - 1) / kPartsAhead;
        if (!all && is_last(v.row_there + v.row_ctas + cta, runs))
          join_rows<HD, kThreads>(out, v, rows, cta, 0, kPartsAhead, runs, sx, sm);
      }
      __syncthreads();
    }
    if (done < n_chunks) {
      at.u = u_end - 1;
      at.next(v);
    }
  }
  cp_wait<0>();
}

template <int HD, int NQ, bool E4M3>
cudaError_t launch_as(const uint16_t* q, uint16_t* o, float scale_log2, const KvView& kv, const SeqView& s, cudaStream_t st) {
  using C = RowsCfg<HD, NQ, E4M3>;
  if (cudaError_t e = allow_shared_memory<attention_rows_kernel<HD, NQ, E4M3>>(C::kBytes)) return e;
  note_launch_begin(kKindAttn, st);
  attention_rows_kernel<HD, NQ, E4M3><<<s.row_ctas, kThreads, C::kBytes, st>>>(q, o, scale_log2, kv, s);
  const cudaError_t e = cudaGetLastError();
  note_launch_end(kKindAttn, st);
  return e;
}

}  // namespace

cudaError_t launch_attention_rows(const uint16_t* q, uint16_t* o, float scale, const KvView& kv, const SeqView& s,
                                  cudaStream_t st) {
  const float c = scale * 1.4426950408889634f;
  const bool two = s.row_limit > 8, f8 = kv.type == kKvE4m3;
  if (s.hd == 128) {
    if (two) return f8 ? launch_as<128, 2, true>(q, o, c, kv, s, st) : launch_as<128, 2, false>(q, o, c, kv, s, st);
    return f8 ? launch_as<128, 1, true>(q, o, c, kv, s, st) : launch_as<128, 1, false>(q, o, c, kv, s, st);
  }
  if (two) return f8 ? launch_as<64, 2, true>(q, o, c, kv, s, st) : launch_as<64, 2, false>(q, o, c, kv, s, st);
  return f8 ? launch_as<64, 1, true>(q, o, c, kv, s, st) : launch_as<64, 1, false>(q, o, c, kv, s, st);
}

}  // namespace mlora
