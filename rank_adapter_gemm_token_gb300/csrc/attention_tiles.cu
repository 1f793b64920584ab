// Attention of sequences with many query rows (chunks of a prompt, whole prompts, groups of many heads) over
// the paged cache, the formula of attention_rows.cu. Bound: the tensor cores and, next to them, the exponentials.
//
// Rows are (token, head of the group) pairs of one key/value head, 256 to a block: all heads of a group share
// its keys. A persistent CTA works on two 128-row tiles at once, so that one tile's softmax runs beside the
// other's products:
//   warps 0-3, 4-7  one softmax warpgroup for each tile, a thread for each row: S from TMEM, running maximum and
//                   sum in base 2, P back to TMEM as 16-bit in place of S, at the end O / sum to global memory.
//                   The maximum moves only when a score passes it by 2^8, so O is rescaled rarely. They also
//                   bring the tile's query rows to shared memory.
//   warps 8-11      keys and values of 128 tokens at a time into a ring of shared-memory tiles. bf16: one warp
//                   issues TMA boxes of whole pages (a lane for each page). e4m3: all four copy codes by cp.async
//                   into a ring of their own and turn them into f16 (exact) in the tiles; each thread converts
//                   what it copied, so no barrier lies between.
//   warp 12         one thread issues tcgen05.mma: S = Q K^T (both from shared memory, K-major) and O += P V with
//                   P from TMEM and V as the N-major operand. TMEM: S/P 2 x 128 columns, O 2 x hd columns.
// e4m3: the key scale multiplies the score, log2 of the value scale is added to it (P then is the weight times the
// scale, at most 2^8 whatever the scales), the sum takes P / value scale; query rows are divided by their largest
// element so that f16 holds them.
// Work: (block, key/value head) items of 128-key tiles one after another, an equal share to each CTA (Shares);
// parts of a split item are joined in key order by the CTA that comes last.
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

constexpr int kThreads = 512;               // 128 registers each at launch, shared out again by role: 184, 80, 64
constexpr int kKeys = kTileKeys;              // 128
constexpr int kHalf = kKeys * 128;            // bytes of 128 rows of 64 16-bit elements (one swizzled half tile)
constexpr float kLazy = 8.0f;                 // log2 of the largest P
constexpr int kSnap = 2;

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
  static constexpr int kBytes = kBarOff + 512 + 1024;
};

// tcgen05.mma with A from TMEM.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Shared-memory descriptor of an N-major operand: rows (keys) of 128 bytes holding 64 elements of N, 128-byte
// swizzle; 8-row groups 1024 bytes apart, the next 64 elements of N one half tile further.
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(kHalf >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
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
// Barrier of tile w's softmax warpgroup.
__device__ __forceinline__ void tile_sync(int w) {
  if (w == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
  else asm volatile("bar.sync 2, 128;" ::: "memory");
}
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

// One item (256-row block, key/value head) and the part [ka, kb) of its key tiles that this CTA takes.
struct Item {
  int blk, kvh, tiles;          // block, head, key tiles of the whole item
  int ka, kb;
  int s, r0, n, len, first, base, rows;
  int end[2];                   // key tiles that tile w of the block works on: [ka, end[w])
  const int32_t* table;
  __device__ __forceinline__ bool present(int w) const { return r0 + 128 * w < rows; }
};

// The CTA's walk over its share of the items; every role runs its own copy.
struct Walk {
  Shares sh;
  int64_t x, x1;                // next unit, end of the share
  Item it;
  __device__ __forceinline__ void block(const SeqView& v, int j) {
    it.blk = j;
    it.s = v.blk_seq[j];
    it.r0 = v.blk_row[j];
    it.n = v.n[it.s];
    it.len = v.len[it.s];
    it.first = v.start[it.s];
    it.table = v.table + static_cast<size_t>(it.s) * v.max_pages;
    it.base = it.len - it.n;
    it.rows = it.n * v.G;
    it.tiles = static_cast<int>((v.blk_pre[j + 1] - v.blk_pre[j]) / v.Hkv);
  }
  __device__ __forceinline__ int64_t cut(const SeqView& v, int J, int64_t c) {
    const int64_t y = sh.raw(c);
    if (y >= sh.total) return sh.total;
    const int j = last_at_most(v.blk_pre, J, y);
    const int64_t p = v.blk_pre[j];
    const int tiles = static_cast<int>((v.blk_pre[j + 1] - p) / v.Hkv);
    const int64_t a = p + static_cast<int64_t>(static_cast<int>(y - p) / tiles) * tiles;
    return sh.snapped(y, a, a + tiles);
  }
  __device__ __forceinline__ bool begin(const SeqView& v) {
    const int J = v.counts[0];
    sh.total = J > 0 ? v.blk_pre[J] : 0;
    if (sh.total == 0) return false;
    sh.n = static_cast<int>(min(static_cast<int64_t>(gridDim.x), sh.total));
    sh.snap = kSnap;
    if (static_cast<int>(blockIdx.x) >= sh.n) return false;
    x = cut(v, J, blockIdx.x);
    x1 = cut(v, J, blockIdx.x + 1);
    if (x >= x1) return false;
    block(v, last_at_most(v.blk_pre, J, x));
    const int rel = static_cast<int>(x - v.blk_pre[it.blk]);
    it.kvh = rel / it.tiles;
    part(v, rel - it.kvh * it.tiles);
    return true;
  }
  __device__ __forceinline__ void part(const SeqView& v, int ka) {
    it.ka = ka;
    it.kb = static_cast<int>(min(static_cast<int64_t>(it.tiles), ka + (x1 - x)));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int last = (min(it.r0 + 128 * (w + 1), it.rows) - 1) / v.G;
      const int need = (it.base + last) / kKeys + 1;
      it.end[w] = it.present(w) ? min(it.kb, need) : it.ka;
      if (it.end[w] < it.ka) it.end[w] = it.ka;
    }
  }
  // Moves to the next item of the share; false at its end.
  __device__ __forceinline__ bool next(const SeqView& v) {
    x += it.kb - it.ka;
    if (x >= x1) return false;
    if (++it.kvh == v.Hkv) {
      it.kvh = 0;
      block(v, it.blk + 1);
    }
    part(v, 0);
    return true;
  }
};

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
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* sc_full = o_full + 2;                     // [kScaleBufs]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sc_full + C::kScaleBufs);
  int* last_sh = reinterpret_cast<int*>(tmem_slot + 2);   // [2]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* err = v.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      ptx::mbar_init(&kv_full[i], E4M3 ? 128 : 1);
      ptx::mbar_init(&kv_empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      ptx::mbar_init(&q_full[w], 128);
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
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;                   // S/P of tile w at 128 w, O at 256 + 128 w

  Walk walk;
  const bool any = walk.begin(v);
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !ptx::mbar_wait(bar, parity, err)) dead = true;
  };

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax of tile w
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int w = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
    uint32_t n_s = 0, n_o = 0;                        // waits done on s_full, o_full
    uint32_t n_sc = 0;                                // key tiles of the CTA so far (scale buffers)
    for (bool go = any; go; go = walk.next(v)) {
      const Item& it = walk.it;
      const int r = it.r0 + 128 * w + row;
      const bool valid = r < it.rows;
      const int tok = valid ? r / v.G : 0;
      const int64_t at = (static_cast<int64_t>(it.first + tok) * v.Hq + it.kvh * v.G + (valid ? r - tok * v.G : 0)) * HD;
      const int lim = valid ? it.base + tok : -1;
      const int first_lim = it.base + (it.r0 + 128 * w) / v.G;      // of the tile's first row: no key past it is free of masks
      float c = scale_log2;
      const int end = it.end[w];
      if (end > it.ka) {
        uint8_t* dst = smem + C::kQ + w * C::kTile + row * 128;
        uint4 x[HD / 8];
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          x[i] = valid ? *reinterpret_cast<const uint4*>(q + at + i * 8) : make_uint4(0u, 0u, 0u, 0u);
        if (E4M3) {
          float most = 0.f;
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            const uint32_t* p = &x[i].x;
#pragma unroll
            for (int k = 0; k < 4; ++k) most = fmaxf(most, fmaxf(fabsf(ptx::bf16_lo(p[k])), fabsf(ptx::bf16_hi(p[k]))));
          }
          if (!(most > 0.f)) most = 1.f;
          const float inv = 1.0f / most;
          c *= most;
#pragma unroll
          for (int i = 0; i < HD / 8; ++i) {
            uint32_t* p = &x[i].x;
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = pack_f16(ptx::bf16_lo(p[k]) * inv, ptx::bf16_hi(p[k]) * inv);
          }
        }
#pragma unroll
        for (int i = 0; i < HD / 8; ++i)
          *reinterpret_cast<uint4*>(dst + (i >> 3) * kHalf + (((i & 7) ^ (row & 7)) * 16)) = x[i];
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&q_full[w]);
      }
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
        float s[kKeys];
        uint32_t(&u)[4][32] = *reinterpret_cast<uint32_t(*)[4][32]>(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) ptx::tmem_ld_32x32b_x32(ts + 32 * i, u[i]);
        ptx::tmem_ld_wait();
        if (E4M3) {
#pragma unroll
          for (int i = 0; i < kKeys; i += 4) {
            const float4 ks = *reinterpret_cast<const float4*>(sc + i);
            const float4 lv = *reinterpret_cast<const float4*>(sc + kKeys + i);
            s[i] = fmaf(s[i] * ks.x, c, lv.x);
            s[i + 1] = fmaf(s[i + 1] * ks.y, c, lv.y);
            s[i + 2] = fmaf(s[i + 2] * ks.z, c, lv.z);
            s[i + 3] = fmaf(s[i + 3] * ks.w, c, lv.w);
          }
        }
        if ((j + 1) * kKeys - 1 > first_lim) {
          const int k = lim - j * kKeys;              // keys 0 .. k of the tile are visible
#pragma unroll
          for (int i = 0; i < kKeys; ++i) s[i] = i > k ? -INFINITY : s[i];
        }
        float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kKeys; i += 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) t4[k] = fmaxf(t4[k], s[i + k]);
        }
        float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        if (!E4M3) top *= c;
        if (j == it.ka) {
          m = top;
        } else if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float up = top > m + kLazy ? top : m;
          const float f = up == m ? 1.f : exp2_approx(m - up);
          m = up;
          l *= f;
#pragma unroll
          for (int i = 0; i < HD / 32; ++i) {
            uint32_t y[32];
            ptx::tmem_ld_32x32b_x32(to + 32 * i, y);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f);
            tmem_st_x32(to + 32 * i, y);
          }
          tmem_st_wait();
        }
        const float mm = m == -INFINITY ? 0.f : m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 64 * h + 2 * i + k;
              s[e] = exp2_approx(E4M3 ? s[e] - mm : fmaf(s[e], c, -mm));
            }
            const int e = 64 * h + 2 * i;
            if (E4M3) {
              const float4 rv = *reinterpret_cast<const float4*>(sc + 2 * kKeys + e);
              sum[0] = fmaf(s[e], rv.x, sum[0]);
              sum[1] = fmaf(s[e + 1], rv.y, sum[1]);
              sum[2] = fmaf(s[e + 2], rv.z, sum[2]);
              sum[3] = fmaf(s[e + 3], rv.w, sum[3]);
              p[i] = pack_f16(s[e], s[e + 1]);
              p[i + 1] = pack_f16(s[e + 2], s[e + 3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) sum[k] += s[e + k];
              p[i] = pack_bf16(s[e], s[e + 1]);
              p[i + 1] = pack_bf16(s[e + 2], s[e + 3]);
            }
          }
          tmem_st_x32(ts + 32 * h, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
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
        const int64_t a = v.blk_pre[it.blk] + static_cast<int64_t>(it.kvh) * it.tiles;
        int c0, cuts;
        walk.sh.inside(a, a + it.tiles, &c0, &cuts);
        if (cuts == 0) {
          const float inv = l > 0.f ? 1.0f / l : l == 0.f ? 0.f : l;
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
                *reinterpret_cast<uint4*>(o + at + 32 * i + 8 * k) = z;
              }
            }
          }
        } else {
          // a part: sums and maximum to the workspace, [slot][tile][hd / 4][row] float4 and [2][row]
          constexpr int64_t kSlot = static_cast<int64_t>(128) * (HD + 2);
          float* parts = v.tile_part;
          auto slot_of = [&](int k) { return parts + ((2 * static_cast<int64_t>(c0 + k) + (k == 0)) * 2 + w) * kSlot; };
          float* mine = slot_of(static_cast<int>(blockIdx.x) - c0);
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
          __threadfence();
          tile_sync(w);
          if (row == 0) last_sh[w] = atomicAdd(&v.tile_sync[2 * c0 + w], 1u) == static_cast<uint32_t>(cuts);
          tile_sync(w);
          if (last_sh[w]) {
            __threadfence();
            float top = -INFINITY, total = 0.f;
            for (int k = 0; k <= cuts; ++k) top = fmaxf(top, __ldcg(slot_of(k) + 128 * HD + row));
            for (int k = 0; k <= cuts; ++k) {
              const float mk = __ldcg(slot_of(k) + 128 * HD + row);
              if (mk != -INFINITY) total = fmaf(exp2_approx(mk - top), __ldcg(slot_of(k) + 128 * HD + 128 + row), total);
            }
            const float inv = total > 0.f ? 1.0f / total : total == 0.f ? 0.f : total;
#pragma unroll 1
            for (int i = 0; i < HD / 16; ++i) {
              float y[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = 0.f;
              for (int k = 0; k <= cuts; ++k) {
                const float* p = slot_of(k);
                const float mk = __ldcg(p + 128 * HD + row);
                if (mk == -INFINITY) continue;
                const float f = exp2_approx(mk - top) * inv;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 z = __ldcg(reinterpret_cast<const float4*>(p) + (4 * i + e) * 128 + row);
                  y[4 * e] = fmaf(f, z.x, y[4 * e]);
                  y[4 * e + 1] = fmaf(f, z.y, y[4 * e + 1]);
                  y[4 * e + 2] = fmaf(f, z.z, y[4 * e + 2]);
                  y[4 * e + 3] = fmaf(f, z.w, y[4 * e + 3]);
                }
              }
              if (valid) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  *reinterpret_cast<uint4*>(o + at + 16 * i + 8 * e) =
                      make_uint4(pack_bf16(y[8 * e], y[8 * e + 1]), pack_bf16(y[8 * e + 2], y[8 * e + 3]),
                                 pack_bf16(y[8 * e + 4], y[8 * e + 5]), pack_bf16(y[8 * e + 6], y[8 * e + 7]));
              }
            }
            if (row == 0) v.tile_sync[2 * c0 + w] = 0;
          }
          tile_sync(w);
        }
      }
      ptx::tc_fence_before();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ keys and values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (!E4M3) {
      if (warp == 8) {
        const int box = min(kv.page, kKeys), boxes = kKeys / box;
        uint32_t n = 0;                               // tiles brought so far
        for (bool go = any; go; go = walk.next(v)) {
          const Item& it = walk.it;
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
      Walk ahead = walk;
      bool more = any;
      int aj = any ? ahead.it.ka : 0, ah = 0;         // next tile to load: key tile, keys (0) or values (1)
      uint32_t n_ld = 0;
      auto load = [&]() {
        if (more) {
          const Item& it = ahead.it;
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
              more = ahead.next(v);
              aj = more ? ahead.it.ka : 0;
            }
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll
      for (int i = 0; i < C::kStages - 1; ++i) load();
      uint32_t n = 0;
      for (bool go = any; go; go = walk.next(v)) {
        const Item& it = walk.it;
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
    // ------------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const uint32_t id_s = idesc16(E4M3, 128, kKeys, false), id_o = idesc16(E4M3, 128, HD, true);
    uint32_t n = 0;                                   // ring position of the item's first key tile
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
    for (bool go = any && warp == 12; go; go = walk.next(v)) {
      const Item& it = walk.it;
      for (int j = it.ka; j <= it.kb; ++j) {
        const uint32_t nk = n + 2 * (j - it.ka), nv = nk - 1;      // ring positions of K_j and V_{j-1}
        if (j > it.ka) {
          const int st = nv % C::kRing;
          wait(&kv_full[st], (nv / C::kRing) & 1);
          const int cut = it.len - (j - 1) * kKeys;
          if (!E4M3 && cut < kKeys) {                 // value rows past the length
            uint8_t* t = smem + C::kRingOff + st * C::kTile;
            for (int r = cut; r < kKeys; ++r)
              if (lane < HD / 8) *reinterpret_cast<uint4*>(t + (lane >> 3) * kHalf + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            ptx::fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (j < it.kb) wait(&kv_full[nk % C::kRing], (nk / C::kRing) & 1);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (j > it.ka && j - 1 < it.end[w]) {
            wait(&p_full[w], n_p[w] & 1);
            ++n_p[w];
            ptx::tc_fence_after();
            if (lane == 0) {
              const uint32_t vt = base + C::kRingOff + (nv % C::kRing) * C::kTile;
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                umma_ts(tmem + 256 + 128 * w, tmem + 128 * w + 8 * k, sw128_nmajor_desc(vt + k * 2048), id_o,
                        j - 1 > it.ka || k > 0);
              if (j == it.end[w]) ptx::umma_commit(&o_full[w]);
            }
          }
          if (j < it.end[w]) {
            if (j == it.ka) {
              wait(&q_full[w], n_q[w] & 1);
              ++n_q[w];
              ptx::tc_fence_after();
            }
            if (lane == 0) {
              const uint32_t qt = base + C::kQ + w * C::kTile, kt = base + C::kRingOff + (nk % C::kRing) * C::kTile;
#pragma unroll
              for (int k = 0; k < kSteps; ++k) {
                const uint32_t off = (k >> 2) * kHalf + (k & 3) * 32;
                ptx::umma_bf16(tmem + 128 * w, ptx::sw128_kmajor_desc(qt + off), ptx::sw128_kmajor_desc(kt + off), id_s, k > 0);
              }
              ptx::umma_commit(&s_full[w]);
            }
          }
        }
        if (lane == 0) {
          if (j > it.ka) ptx::umma_commit(&kv_empty[nv % C::kRing]);
          if (j < it.kb) ptx::umma_commit(&kv_empty[nk % C::kRing]);
        }
        __syncwarp();
      }
      n += 2 * (it.kb - it.ka);
    }
  }
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
  attention_tiles_kernel<HD, E4M3><<<s.tile_ctas, kThreads, C::kBytes, st>>>(tk, tv, q, o, scale_log2, kv, s);
  const cudaError_t e = cudaGetLastError();
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
