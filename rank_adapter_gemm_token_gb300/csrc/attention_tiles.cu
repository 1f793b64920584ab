// Attention of sequences with many query rows (chunks of a prompt, whole prompts, groups of many heads) over
// the paged cache, the formula of attention_rows.cu. Bound: the tensor cores and, next to them, the exponentials.
//
// Rows are (token, head of the group) pairs of one key/value head, 256 to a block: all heads of a group share
// its keys. A persistent CTA works on two 128-row tiles at once, so that one tile's softmax runs beside the
// other's products:
//   warps 0-3, 4-7  one softmax warpgroup for each tile, a thread for each row: S from TMEM, running maximum and
//                   sum in base 2, P back to TMEM as 16-bit in place of S, at the end O / sum to global memory.
//                   The maximum moves only when a score passes it by 2^8, so O is rescaled rarely.
//   warps 8-11      keys and values of 128 tokens at a time into a ring of shared-memory tiles. bf16: one warp
//                   issues TMA boxes of whole pages (a lane for each page). e4m3: all four copy codes by cp.async
//                   into a ring of their own and turn them into f16 (exact) in the tiles; each thread converts
//                   what it copied, so no barrier lies between.
//   warp 12         tcgen05.mma: S = Q K^T (both from shared memory, K-major) and O += P V with P from TMEM and V as
//                   the N-major operand. TMEM: S/P 2 x 128 columns, O 2 x hd columns. The instructions are issued
//                   under a predicate in uniform control flow: issued inside a divergent branch each took 120
//                   cycles, twice its execution.
//   warps 13-15     the query rows of the next item, while the last products of this one run.
// e4m3: the key scale multiplies the score, log2 of the value scale is added to it (P then is the weight times the
// scale, at most 2^8 whatever the scales), the sum takes P / value scale; query rows are divided by their largest
// element so that f16 holds them.
// Work: (block, key/value head) items of 128-key tiles one after another, an equal share to each CTA (seq_meta.cu);
// parts of a split item are joined by attention_join.cu.
// Value rows past the cached length are zeroed in shared memory, scores past a row's limit are replaced by -inf:
// what lies there has no effect. Every wait is bounded: after 2 s a role records the timeout, stops waiting and
// runs on to the end.
#include <algorithm>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kThreads = 512;               // 128 registers each at launch, shared out again by role: 168, 96, 80
constexpr int kKeys = kTileKeys;              // 128
constexpr int kHalf = kKeys * 128;            // bytes of 128 rows of 64 16-bit elements (one swizzled half tile)
constexpr float kLazy = 8.0f;                 // log2 of the largest P
constexpr int kQThreads = 96;                 // threads that bring the query rows

template <int HD, bool E4M3>
struct TilesCfg {
  static constexpr int kHalves = HD / 64;
  static constexpr int kTile = kHalves * kHalf;
  static constexpr int kRing = E4M3 ? 3 : (HD == 128 ? 4 : 6);     // 16-bit key / value tiles
  static constexpr int kCodes = kKeys * HD;                        // e4m3 bytes of a tile
  static constexpr int kStages = HD == 128 ? 3 : 6;                // tiles of codes on their way
  static constexpr int kSegs = HD / 16;                            // 16-byte segments of a row of codes
  static constexpr int kScaleBufs = 4;
  static constexpr int kQ = 0;
  static constexpr int kRingOff = 2 * kTile;
  static constexpr int kCodeOff = kRingOff + kRing * kTile;
  static constexpr int kRawScaleOff = kCodeOff + (E4M3 ? kStages * kCodes : 0);  // scales on their way: [kStages][2][128]
  static constexpr int kScaleOff = kRawScaleOff + (E4M3 ? kStages * 2 * kKeys * 4 : 0);   // [kScaleBufs][3][128] floats
  static constexpr int kBarOff = kScaleOff + (E4M3 ? kScaleBufs * 3 * kKeys * 4 : 0);
  static constexpr int kQScaleOff = kBarOff + 512;                 // e4m3: [2][tile][128] scales of the query rows
  static constexpr int kWalkOff = kQScaleOff + (E4M3 ? 2 * 2 * 128 * 4 : 0);
  static constexpr int kBytes = kWalkOff + 20 * 128 + 1024;
};

// tcgen05.mma, A from shared memory or from TMEM, and the commit, for the lane whose `on` is set.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void umma_commit_on(uint64_t* bar, uint32_t on) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(ptx::smem_u32(bar)), "r"(on)
      : "memory");
}
// Shared-memory descriptors (128-byte swizzle, 8-row groups 1024 bytes apart) without the address: the K-major form of
// ptx::sw128_kmajor_desc, and an N-major operand: rows (keys) of 128 bytes holding 64 elements of N, the next 64 one half
// tile further. Addresses (in 16 bytes) are added; shared memory ends before their field does.
constexpr uint64_t kDescK = (uint64_t(1) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
constexpr uint64_t kDescN = (uint64_t(kHalf >> 4) << 16) | (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
// Instruction descriptor of kind::f16 (fp32 D; A and B bf16, or f16), B N-major on request.
__host__ __device__ constexpr uint32_t idesc16(bool f16, int M, int N, bool b_nmajor) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_nmajor ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair_u(uint32_t x, uint32_t y) { return pair(__uint_as_float(x), __uint_as_float(y)); }

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, bool full) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(full ? 4 : 0) : "memory");
}

// The CTA's walk over its share of the items (256-row block, key/value head), with the part [ka, kb) of the item's key
// tiles that the CTA takes. Every role walks on its own.
struct alignas(128) Walk {
  int left;                     // units left in the share
  int blk, kvh;
  int ka, kb, tiles;
  int n, len, first, r0;        // the block's sequence, and its first row
  int base, rows;               // position of the sequence's first new token; its rows
  int end[2];                   // tile w of the block works on key tiles [ka, end[w])
  const int32_t* table;
  __device__ __forceinline__ bool present(int w) const { return r0 + 128 * w < rows; }
  __device__ __forceinline__ bool whole() const { return ka == 0 && kb == tiles; }
  __device__ __forceinline__ void block(const SeqView& v) {
    const TileBlk b = v.blk[blk];
    n = b.n, len = b.len, first = b.start, r0 = b.r0, tiles = b.tiles;
    table = v.table + static_cast<size_t>(b.seq) * v.max_pages;
    base = len - n;
    rows = n * v.G;
  }
  __device__ __forceinline__ void part(const SeqView& v, int from) {
    ka = from;
    kb = min(tiles, ka + left - (ka == 0 ? kTileHead : 0));       // (a cut inside an item lies past its head)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int last = (min(r0 + 128 * (w + 1), rows) - 1) / v.G;
      end[w] = present(w) ? max(ka, min(kb, (base + last) / kKeys + 1)) : ka;
    }
  }
  __device__ __forceinline__ bool begin(const SeqView& v) {
    const int4 s = *reinterpret_cast<const int4*>(v.tile_share + blockIdx.x);
    left = s.w;
    if (left <= 0) return false;
    blk = s.x, kvh = s.y;
    block(v);
    part(v, s.z);
    return true;
  }
  __device__ __forceinline__ bool next(const SeqView& v) {
    left -= kb - ka + (ka == 0 ? kTileHead : 0);
    if (left <= 0) return false;
    if (++kvh == v.Hkv) {
      kvh = 0;
      ++blk;
      block(v);
    }
    part(v, 0);
    return true;
  }
};
static_assert(sizeof(Walk) <= 128, "a walk's place in shared memory");

template <int HD, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
attention_tiles_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const uint16_t* __restrict__ q, uint16_t* __restrict__ o, float scale_log2, KvView kv, SeqView v) {
  using C = TilesCfg<HD, E4M3>;
  constexpr int kSteps = HD / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_u32(smem);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* kv_empty = kv_full + C::kRing;
  uint64_t* q_full = kv_empty + C::kRing;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* sc_full = o_full + 2;                     // [kScaleBufs]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_full + C::kScaleBufs);
  float* q_scale = reinterpret_cast<float*>(smem + C::kQScaleOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* err = v.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      ptx::mbar_init(&kv_full[i], E4M3 ? 128 : 1);
      ptx::mbar_init(&kv_empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      ptx::mbar_init(&q_full[w], kQThreads);
      ptx::mbar_init(&q_empty[w], 1);
      ptx::mbar_init(&s_full[w], 1);
      ptx::mbar_init(&p_full[w], 128);
      ptx::mbar_init(&o_full[w], 1);
    }
    for (int i = 0; i < C::kScaleBufs; ++i) ptx::mbar_init(&sc_full[i], 128);
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 12) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::grid_dependents_launch();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;                   // S/P of tile w at 128 w, O at 256 + 128 w

  // Each warp's walk lives in shared memory, moved by its first lane: the fields are read a few times an item, and
  // a softmax thread has no registers to keep them in.
  Walk* walks = reinterpret_cast<Walk*>(smem + C::kWalkOff);   // [13], and [16 ..]: the loads' own
  Walk& walk = walks[warp];
  bool any;
  {
    Walk first{};
    any = first.begin(v);
    if (lane == 0) walk = first;
    if (lane == 0 && warp >= 8 && warp < 12) walks[warp + 8] = first;
    __syncwarp();
  }
  auto advance = [&](Walk& w) {
    __syncwarp();
    int go = 0;
    if (lane == 0) go = w.next(v);
    go = __shfl_sync(0xffffffffu, go, 0);
    __syncwarp();
    return go != 0;
  };
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !ptx::mbar_wait(bar, parity, err)) dead = true;
  };

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax of tile w
    asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    const int w = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
    uint32_t n_s = 0, n_o = 0;                        // waits done on s_full, o_full
    uint32_t n_sc = 0;                                // key tiles of the CTA so far (scale buffers)
    for (bool go = any; go; go = advance(walk)) {
      const Walk& it = walk;
      const int r = it.r0 + 128 * w + row;
      const bool valid = r < it.rows;
      const int tok = valid ? r / v.G : 0;
      const int lim = valid ? it.base + tok : -1;
      const int first_lim = it.base + (it.r0 + 128 * w) / v.G;      // the tile's first row sees the fewest keys
      float c = scale_log2;
      const int end = it.end[w];
      float m = -INFINITY, l = 0.f;
      for (int j = it.ka; j < end; ++j) {
        const float* sc = nullptr;
        if (E4M3) {
          const uint32_t t = n_sc + (j - it.ka);
          wait(&sc_full[t % C::kScaleBufs], (t / C::kScaleBufs) & 1);
          sc = reinterpret_cast<const float*>(smem + C::kScaleOff) + (t % C::kScaleBufs) * 3 * kKeys;
        }
        wait(&s_full[w], n_s & 1);
        ++n_s;
        ptx::tc_fence_after();
        // (the query rows and their scales were there before the products that s_full stands for)
        if (E4M3 && j == it.ka) c *= q_scale[((n_o & 1) * 2 + w) * 128 + row];
        // Two passes over S, 32 columns at a time: the maximum, then the weights. Reading S from TMEM twice costs
        // less than holding 128 scores in registers (which spilled).
        const bool masked = (j + 1) * kKeys - 1 > first_lim;
        const uint64_t cc = pair(c, c);
        const int seen = lim - j * kKeys;             // keys 0 .. seen of the tile are visible
        auto scores = [&](uint32_t (&x)[32], int h) {  // columns 32 h ...: scaled (e4m3) and masked
          if (E4M3) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 ks = *reinterpret_cast<const float4*>(sc + 32 * h + i);
              const float4 lv = *reinterpret_cast<const float4*>(sc + kKeys + 32 * h + i);
              const float2 y = unpair(fma_pair(mul_pair(pair_u(x[i], x[i + 1]), pair(ks.x, ks.y)), cc, pair(lv.x, lv.y)));
              const float2 z = unpair(fma_pair(mul_pair(pair_u(x[i + 2], x[i + 3]), pair(ks.z, ks.w)), cc, pair(lv.z, lv.w)));
              x[i] = __float_as_uint(y.x), x[i + 1] = __float_as_uint(y.y);
              x[i + 2] = __float_as_uint(z.x), x[i + 3] = __float_as_uint(z.y);
            }
          }
          if (masked) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 32 * h + i > seen ? 0xff800000u : x[i];
          }
        };
        auto largest = [&](const uint32_t (&x)[32], float t) {
          float u = __uint_as_float(x[0]);
#pragma unroll
          for (int i = 1; i < 16; ++i) {
            u = fmaxf(u, __uint_as_float(x[i]));
            t = fmaxf(t, __uint_as_float(x[i + 16]));
          }
          return fmaxf(fmaxf(t, __uint_as_float(x[16])), u);
        };
        uint32_t xa[32], xb[32];
        ptx::tmem_ld_32x32b_x32(ts, xa);
        ptx::tmem_ld_32x32b_x32(ts + 32, xb);
        ptx::tmem_ld_wait();
        scores(xa, 0);
        float top = largest(xa, -INFINITY);
        ptx::tmem_ld_32x32b_x32(ts + 64, xa);
        scores(xb, 1);
        top = largest(xb, top);
        ptx::tmem_ld_wait();
        ptx::tmem_ld_32x32b_x32(ts + 96, xb);
        scores(xa, 2);
        top = largest(xa, top);
        ptx::tmem_ld_wait();
        ptx::tmem_ld_32x32b_x32(ts, xa);
        scores(xb, 3);
        top = largest(xb, top);
        if (!E4M3) top *= c;
        if (j == it.ka) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float up = top > m + kLazy ? top : m;
          const float f = up == m ? 1.f : exp2_approx(m - up);
          m = up;
          l *= f;
          ptx::tmem_ld_wait();                        // the columns read ahead
#pragma unroll 1
          for (int i = 0; i < HD / 32; ++i) {
            ptx::tmem_ld_32x32b_x32(to + 32 * i, xb);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) xb[k] = __float_as_uint(__uint_as_float(xb[k]) * f);
            tmem_st_x32(to + 32 * i, xb);
          }
        }
        const float mm = m == -INFINITY ? 0.f : m;
        const uint64_t neg = pair(-mm, -mm);
        uint64_t sum = 0, sum1 = 0;                   // two zeros each
        auto weights = [&](uint32_t (&x)[32], int h) {
          scores(x, h);
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const uint64_t y0 = pair_u(x[i], x[i + 1]), y1 = pair_u(x[i + 2], x[i + 3]);
            float2 e0 = unpair(E4M3 ? add_pair(y0, neg) : fma_pair(y0, cc, neg));
            float2 e1 = unpair(E4M3 ? add_pair(y1, neg) : fma_pair(y1, cc, neg));
            e0.x = exp2_approx(e0.x), e0.y = exp2_approx(e0.y);
            e1.x = exp2_approx(e1.x), e1.y = exp2_approx(e1.y);
            if (E4M3) {
              const float4 rv = *reinterpret_cast<const float4*>(sc + 2 * kKeys + 32 * h + i);
              sum = fma_pair(pair(e0.x, e0.y), pair(rv.x, rv.y), sum);
              sum1 = fma_pair(pair(e1.x, e1.y), pair(rv.z, rv.w), sum1);
              p[i / 2] = pack_f16(e0.x, e0.y);
              p[i / 2 + 1] = pack_f16(e1.x, e1.y);
            } else {
              sum = add_pair(sum, pair(e0.x, e0.y));
              sum1 = add_pair(sum1, pair(e1.x, e1.y));
              p[i / 2] = pack_bf16(e0.x, e0.y);
              p[i / 2 + 1] = pack_bf16(e1.x, e1.y);
            }
          }
          tmem_st_x16(ts + 16 * h, p);
        };
        ptx::tmem_ld_wait();
        ptx::tmem_ld_32x32b_x32(ts + 32, xb);
        weights(xa, 0);
        ptx::tmem_ld_wait();
        ptx::tmem_ld_32x32b_x32(ts + 64, xa);
        weights(xb, 1);
        ptx::tmem_ld_wait();
        ptx::tmem_ld_32x32b_x32(ts + 96, xb);
        weights(xa, 2);
        ptx::tmem_ld_wait();
        weights(xb, 3);
        const float2 total = unpair(add_pair(sum, sum1));
        l += total.x + total.y;
        tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&p_full[w]);
      }
      n_sc += it.kb - it.ka;
      if (end > it.ka) {
        wait(&o_full[w], n_o & 1);
        ++n_o;
        ptx::tc_fence_after();
      }

      if (it.present(w)) {
        if (it.whole()) {
          const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;      // NaN stays
          uint16_t* dst = o + (static_cast<int64_t>(it.first + tok) * v.Hq + it.kvh * v.G + (r - tok * v.G)) * HD;
#pragma unroll
          for (int i = 0; i < HD / 32; ++i) {
            uint32_t y[32];
            ptx::tmem_ld_32x32b_x32(to + 32 * i, y);
            ptx::tmem_ld_wait();
            if (valid) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint4 z;
                z.x = pack_bf16(__uint_as_float(y[8 * k]) * inv, __uint_as_float(y[8 * k + 1]) * inv);
                z.y = pack_bf16(__uint_as_float(y[8 * k + 2]) * inv, __uint_as_float(y[8 * k + 3]) * inv);
                z.z = pack_bf16(__uint_as_float(y[8 * k + 4]) * inv, __uint_as_float(y[8 * k + 5]) * inv);
                z.w = pack_bf16(__uint_as_float(y[8 * k + 6]) * inv, __uint_as_float(y[8 * k + 7]) * inv);
                *reinterpret_cast<uint4*>(dst + 32 * i + 8 * k) = z;
              }
            }
          }
        } else {
          float* mine = v.tile_part + ((2 * static_cast<int64_t>(blockIdx.x) + (it.ka == 0)) * 2 + w) * tile_slot(v);
          if (end > it.ka) {
#pragma unroll
            for (int i = 0; i < HD / 32; ++i) {
              uint32_t y[32];
              ptx::tmem_ld_32x32b_x32(to + 32 * i, y);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k)
                reinterpret_cast<uint4*>(mine)[(8 * i + k) * 128 + row] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            }
          }
          mine[128 * HD + row] = m;
          mine[128 * HD + 128 + row] = l;
        }
      }
      ptx::tc_fence_before();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ keys and values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (!E4M3) {
      if (warp == 8) {
        const int box = min(kv.page, kKeys), boxes = kKeys / box;
        uint32_t n = 0;                               // tiles brought so far
        for (bool go = any; go; go = advance(walk)) {
          const Walk& it = walk;
          for (int j = it.ka; j < it.kb; ++j) {
            const int key = j * kKeys + lane * box;
            const bool mine = lane < boxes && key < it.len;
            int at = 0;
            if (mine) at = ((it.table[key >> kv.page_log2] * v.Hkv + it.kvh) << kv.page_log2) + (key & (kv.page - 1));
            const int count = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll
            for (int h = 0; h < 2; ++h, ++n) {        // the keys, then the values
              const int st = n % C::kRing;
              wait(&kv_empty[st], ((n / C::kRing) & 1) ^ 1);
              uint8_t* dst = smem + C::kRingOff + st * C::kTile + lane * box * 128;
              if (lane == 0) ptx::mbar_arrive_expect_tx(&kv_full[st], count * box * 128 * C::kHalves);
              __syncwarp();
              if (mine) {
#pragma unroll
                for (int x = 0; x < C::kHalves; ++x)
                  ptx::tma_load_2d(dst + x * kHalf, h ? &tmap_v : &tmap_k, &kv_full[st], 64 * x, at);
              }
            }
          }
        }
        // the copies of an abandoned run are waited for by the kernel's end
      }
    } else {
      const int tid = threadIdx.x - 256;
      constexpr int kStep = 128 / C::kSegs;           // rows of one copy of all threads
      constexpr int kCopies = kKeys / kStep;
      const int seg = tid % C::kSegs, r_in = tid / C::kSegs;
      const uint32_t codes = base + C::kCodeOff + tid * 16;
      const uint32_t raw = base + C::kRawScaleOff + tid * 4;
      // loads run kStages - 1 tiles ahead of the conversion, over a walk of their own
      Walk& ahead = walks[warp + 8];
      bool more = any;
      int aj = any ? ahead.ka : 0, ah = 0;         // next tile to load: key tile, keys (0) or values (1)
      uint32_t n_ld = 0;
      auto load = [&]() {
        if (more) {
          const Walk& it = ahead;
          const int st = n_ld % C::kStages;
          const uint8_t* src = static_cast<const uint8_t*>(ah ? kv.V : kv.K);
#pragma unroll
          for (int i = 0; i < kCopies; ++i) {
            const int key = aj * kKeys + i * kStep + r_in;
            const bool in = key < it.len;
            const int page = it.table[min(key, it.len - 1) >> kv.page_log2];
            const int64_t at = ((static_cast<int64_t>(page) * v.Hkv + it.kvh) << kv.page_log2) + (key & (kv.page - 1));
            cp16(codes + st * C::kCodes + i * 2048, src + at * HD + seg * 16, in);
          }
          {
            const int key = aj * kKeys + tid;
            const bool in = key < it.len;
            const int page = it.table[min(key, it.len - 1) >> kv.page_log2];
            const int64_t at = ((static_cast<int64_t>(page) * v.Hkv + it.kvh) << kv.page_log2) + (key & (kv.page - 1));
            if (ah == 0) {                            // both scales come with the keys: the scores need them
              cp4(raw + st * 2 * kKeys * 4, kv.k_scale + at, in);
              cp4(raw + st * 2 * kKeys * 4 + kKeys * 4, kv.v_scale + at, in);
            }
          }
          ++n_ld;
          if (ah == 0) {
            ah = 1;
          } else {
            ah = 0;
            if (++aj == it.kb) {
              more = advance(ahead);
              aj = more ? ahead.ka : 0;
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int i = 0; i < C::kStages - 1; ++i) load();
      uint32_t n = 0;
      for (bool go = any; go; go = advance(walk)) {
        const Walk& it = walk;
        for (int j = it.ka; j < it.kb; ++j) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h, ++n) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
            const int st = n % C::kRing, cs = n % C::kStages;
            wait(&kv_empty[st], ((n / C::kRing) & 1) ^ 1);
            if (h == 0) {
              const uint32_t t = n / 2;
              float* sc = reinterpret_cast<float*>(smem + C::kScaleOff) + (t % C::kScaleBufs) * 3 * kKeys + tid;
              const float* rw = reinterpret_cast<const float*>(smem + C::kRawScaleOff) + cs * 2 * kKeys + tid;
              const float ks = rw[0], vs = rw[kKeys];
              sc[0] = ks;
              sc[kKeys] = __log2f(vs);
              sc[2 * kKeys] = vs > 0.f ? __fdividef(1.0f, vs) : 0.f;      // a NaN scale counts in the exponent alone
              ptx::mbar_arrive(&sc_full[t % C::kScaleBufs]);
            }
            uint8_t* dst = smem + C::kRingOff + st * C::kTile + (seg >> 2) * kHalf;
            const uint8_t* src = smem + C::kCodeOff + tid * 16 + cs * C::kCodes;
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
              const uint4 cd = *reinterpret_cast<const uint4*>(src + i * 2048);
              const uint4 lo = make_uint4(e4m3x2_f16x2(cd.x), e4m3x2_f16x2(cd.x >> 16), e4m3x2_f16x2(cd.y), e4m3x2_f16x2(cd.y >> 16));
              const uint4 hi = make_uint4(e4m3x2_f16x2(cd.z), e4m3x2_f16x2(cd.z >> 16), e4m3x2_f16x2(cd.w), e4m3x2_f16x2(cd.w >> 16));
              const int r = i * kStep + r_in, p = (seg & 3) * 2;
              const bool odd = seg >= 4;              // the halves' lanes take different banks
              *reinterpret_cast<uint4*>(dst + r * 128 + (((p + (odd ? 1 : 0)) ^ (r & 7)) * 16)) = odd ? hi : lo;
              *reinterpret_cast<uint4*>(dst + r * 128 + (((p + (odd ? 0 : 1)) ^ (r & 7)) * 16)) = odd ? lo : hi;
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&kv_full[st]);
            load();
          }
        }
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 12) {
    // ------------------------------------------------------------------ products
    const uint32_t id_s = idesc16(E4M3, 128, kKeys, false), id_o = idesc16(E4M3, 128, HD, true);
    const uint32_t on = lane == 0;
    uint32_t n = 0;                                   // ring position of the item's first key tile
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
    for (bool go = any; go; go = advance(walk)) {
      const int ka = walk.ka, kb = walk.kb, len = walk.len;
      const int end[2] = {walk.end[0], walk.end[1]};
      for (int j = ka; j <= kb; ++j) {
        const uint32_t nk = n + 2 * (j - ka), nv = nk - 1;         // ring positions of K_j and V_{j-1}
        const uint32_t vs = nv % C::kRing, ks = nk % C::kRing;
        if (j > ka) {
          wait(&kv_full[vs], (nv / C::kRing) & 1);
          const int cut = len - (j - 1) * kKeys;
          if (!E4M3 && cut < kKeys) {                 // value rows past the length
            uint8_t* t = smem + C::kRingOff + vs * C::kTile;
            for (int r = cut; r < kKeys; ++r)
              if (lane < HD / 8) *reinterpret_cast<uint4*>(t + (lane >> 3) * kHalf + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (j < kb) wait(&kv_full[ks], (nk / C::kRing) & 1);
        const uint64_t dv = kDescN + ((base + C::kRingOff + vs * C::kTile) >> 4);
        const uint64_t dk = kDescK + ((base + C::kRingOff + ks * C::kTile) >> 4);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (j > ka && j - 1 < end[w]) {
            wait(&p_full[w], n_p[w] & 1);
            ++n_p[w];
            ptx::tc_fence_after();
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              umma_ts(tmem + 256 + 128 * w, tmem + 128 * w + 8 * k, dv + k * (2048 >> 4), id_o, j - 1 > ka || k > 0, on);
            if (j == end[w]) umma_commit_on(&o_full[w], on);
          }
          if (j < end[w]) {
            if (j == ka) {
              wait(&q_full[w], n_q[w] & 1);
              ++n_q[w];
              ptx::tc_fence_after();
            }
            const uint64_t dq = kDescK + ((base + C::kQ + w * C::kTile) >> 4);
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
              const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
              umma_ss(tmem + 128 * w, dq + off, dk + off, id_s, k > 0, on);
            }
            umma_commit_on(&s_full[w], on);
            if (j + 1 == end[w]) umma_commit_on(&q_empty[w], on);
          }
        }
        if (j > ka) umma_commit_on(&kv_empty[vs], on);
        if (j < kb) umma_commit_on(&kv_empty[ks], on);
      }
      n += 2 * (kb - ka);
    }
    } else {
    // ------------------------------------------------------------------ queries
    const int tid = threadIdx.x - 13 * 32;
    uint32_t n_q[2] = {0, 0};
    for (bool go = any; go; go = advance(walk)) {
      const Walk& it = walk;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (it.end[w] <= it.ka) continue;
        wait(&q_empty[w], (n_q[w] & 1) ^ 1);
        uint8_t* tile = smem + C::kQ + w * C::kTile;
        const int r0 = it.r0 + 128 * w, rows = it.rows;
        const uint16_t* src = q + (static_cast<int64_t>(it.first) * v.Hq + it.kvh * v.G) * HD;
        if (!E4M3) {
          constexpr int kRowSegs = HD / 8;
          for (int i = tid; i < 128 * kRowSegs; i += kQThreads) {
            const int row = i / kRowSegs, seg = i % kRowSegs, r = r0 + row;
            const int tok = r < rows ? r / v.G : 0;
            cp16(base + C::kQ + w * C::kTile + (seg >> 3) * kHalf + row * 128 + (((seg & 7) ^ (row & 7)) * 16),
                 src + (static_cast<int64_t>(tok) * v.Hq + (r < rows ? r - tok * v.G : 0)) * HD + seg * 8, r < rows);
          }
          asm volatile("cp.async.commit_group;" ::: "memory");
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        } else {
          for (int row = tid; row < 128; row += kQThreads) {
            const int r = r0 + row, tok = r < rows ? r / v.G : 0;
            const uint4* x = reinterpret_cast<const uint4*>(src + (static_cast<int64_t>(tok) * v.Hq + (r < rows ? r - tok * v.G : 0)) * HD);
            float most = 0.f;
#pragma unroll 8
            for (int i = 0; i < HD / 8; ++i) {
              const uint4 y = __ldg(x + i);
              const uint32_t p[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) most = fmaxf(most, fmaxf(fabsf(ptx::bf16_lo(p[k])), fabsf(ptx::bf16_hi(p[k]))));
            }
            if (!(most > 0.f)) most = 1.f;
            const float inv = r < rows ? 1.0f / most : 0.f;
#pragma unroll 8
            for (int i = 0; i < HD / 8; ++i) {
              const uint4 y = __ldg(x + i);
              uint32_t p[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) p[k] = r < rows ? pack_f16(ptx::bf16_lo(p[k]) * inv, ptx::bf16_hi(p[k]) * inv) : 0u;
              *reinterpret_cast<uint4*>(tile + (i >> 3) * kHalf + row * 128 + (((i & 7) ^ (row & 7)) * 16)) = make_uint4(p[0], p[1], p[2], p[3]);
            }
            q_scale[((n_q[w] & 1) * 2 + w) * 128 + row] = most;
          }
        }
        ++n_q[w];
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&q_full[w]);
      }
    }
  }
  }
  ptx::grid_dependency_wait();                        // this grid's end stands for the row kernel's too
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool E4M3>
cudaError_t launch_as(const CUtensorMap& tk, const CUtensorMap& tv, const uint16_t* q, uint16_t* o, float scale_log2,
                      const KvView& kv, const SeqView& s, cudaStream_t st) {
  using C = TilesCfg<HD, E4M3>;
  static cudaError_t once = cudaFuncSetAttribute(attention_tiles_kernel<HD, E4M3>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (once != cudaSuccess) return once;
  note_launch_begin(kKindAttn, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(s.tile_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attention_tiles_kernel<HD, E4M3>, tk, tv, q, o, scale_log2, kv, s);
  note_launch_end(kKindAttn, st);
  return e;
}

}  // namespace

bool make_kv_maps(const KvView& kv, CUtensorMap* k, CUtensorMap* v) {
  const long rows = static_cast<long>(kv.n_pages) * kv.page * kv.Hkv;
  const int box = std::min(kv.page, kTileKeys);
  return make_tmap_bf16(k, kv.K, rows, kv.hd, box, 64) && make_tmap_bf16(v, kv.V, rows, kv.hd, box, 64);
}

cudaError_t launch_attention_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const uint16_t* q, uint16_t* o,
                                   float scale, const KvView& kv, const SeqView& s, cudaStream_t st) {
  const float c = scale * 1.4426950408889634f;
  const bool f8 = kv.type == kKvE4m3;
  if (s.hd == 128)
    return f8 ? launch_as<128, true>(tk, tv, q, o, c, kv, s, st) : launch_as<128, false>(tk, tv, q, o, c, kv, s, st);
  return f8 ? launch_as<64, true>(tk, tv, q, o, c, kv, s, st) : launch_as<64, false>(tk, tv, q, o, c, kv, s, st);
}

}  // namespace mlora
