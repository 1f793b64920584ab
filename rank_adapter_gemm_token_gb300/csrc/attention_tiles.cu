// Attention of sequences with many query rows (chunks of a prompt, whole prompts, groups of many heads) over
// the paged cache, the formula of attention_rows.cu. Bound: the tensor cores and, next to them, the exponentials.
//
// Rows are (token, head of the group) pairs of one key/value head: all heads of a group share its keys. A tile holds the
// rows of as many whole tokens as fit 128 rows (128 / G), a block two tiles. A persistent CTA works on both tiles of a
// block at once, so that one tile's softmax runs beside the other's products:
//   warps 0-3, 4-7  one softmax warpgroup for each tile, a thread for each row: S from TMEM, running maximum and
//                   sum in base 2, P back to TMEM as 16-bit in place of S, at the end O / sum to global memory.
//                   The maximum moves only when a score passes it by 2^8 (e4m3: 2^4), so O is rescaled rarely.
//   warps 8-11      bf16: the first brings keys and values of 128 tokens at a time into a ring of shared-memory tiles
//                   by TMA boxes of whole pages (a lane for each page), the second clears value rows past the
//                   sequence's length. e4m3: warp 14 brings the codes, all four turn them into f16 in the ring's tiles.
//   warp 12         tcgen05.mma: S = Q K^T (both from shared memory, K-major) and O += P V with P from TMEM and V as
//                   the N-major operand. TMEM: S/P 2 x 128 columns, O 2 x hd columns. One elected thread issues them:
//                   chosen by its lane number instead, each instruction took 120 cycles to issue, twice its execution;
//                   with a warp for each tile, their instructions alternate and the rate falls by a third.
//   warps 15, 13    the next item's queries of one tile each by TMA, while the last products of this one run (e4m3: and
//                   their f16 form).
// e4m3: codes become f16 times their scale's first 7 bits and a power of two, which is exact, so that S is a sum of exact products.
// What is left of the key's scale (1 +- 2^-7) multiplies the score in fp32, to 2^-16, and what is left of the value's (up to
// 1 + 2^-6) the weight, to 2^-14, before its one rounding to f16. (With scales rounded to f16, and the products with the codes again,
// every score of a key was off by up to 2^-10: at scores of 60 its weight by 6 %.) 2^E, the binary power of the tile's largest
// value scale, is added to the scores (P then is the weight times that power, at most 2^15 whatever the scales) and 2^-E
// multiplies the sum. The largest row of a tile is lifted by 64 to the top of f16's range: rows of scales 2^20 below it,
// which may be all that an early token sees of the tile, keep their bits. Query rows are lifted by a power of two, most by the
// same one. So one word a key, from shared memory, is all that the softmax reads, and only where it takes the exponentials:
// the maximum is taken of S without it and raised by its bound (scores above 100 in base 2 are gone through again with it).
// A word read by all lanes of a warp costs the shared memory a cycle and the warp a quarter of an instruction: 8000 tokens took
// 712 us with a factor of the key in both passes and one of the value beside the second, 650 without the first of them, 600 so
// (and 546 with the rounded scales, whose one factor a key came after the exponential).
// Work: (block, key/value head) items of 128-key tiles, dealt out whole or in equal shares, a list for each CTA (seq_meta.cu);
// parts of a split item are joined by attention_join.cu.
// Measured on the GPU, 32 heads of 128 on 8: one prompt of 8000 tokens 331 us, 1580 TFLOP/s, at 2070 MHz (357 us in calls for
// seconds on end, when the power cap holds 1935 MHz; tcgen05 busy for 0.6 to 0.7 of the cycles; the rest is a softmax that its own
// products wait for, TMEM being full with two tiles); 512 tokens on 32000 191 us, 1415; 8 x 512 tokens 32 us, 540: of an item's first
// and last tile about 4400 cycles, 1.5 tiles, overlap with nothing. e4m3: 8000 tokens 600 us, 875; 8 x 512 tokens 50 us.
// Value rows past the cached length are zeroed in shared memory, scores past a row's limit are replaced by -inf:
// what lies there has no effect. Every wait is bounded: after 2 s a role records the timeout, brings no more
// copies and products (its copies are 2 s old by then, its products are waited for), stops waiting and runs on to the end.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "attention.h"
#include "attention.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlora {
namespace {

constexpr int kThreads = 512;               // 128 registers each at launch, shared out again by role (kSoftmaxRegs)
constexpr int kKeys = kTileKeys;              // 128
constexpr int kHalf = kKeys * 128;            // bytes of 128 rows of 64 16-bit elements (one swizzled half tile)
// log2 of the largest exponential; e4m3: and of the factor that lifts P in f16, whose normal numbers then reach down to
// weights of 2^-25 (their values may be that much larger than the others), while P stays at 2^15 at most. (A limit of 4 in place of 8 rescales O more often: 552 us against 548 at 8000 tokens; one of 2 573.)
template <bool E4M3>
constexpr float kLazy = E4M3 ? 4.0f : 8.0f;
template <bool E4M3>
constexpr float kUp = E4M3 ? 11.0f : 0.0f;
constexpr int kLiftLog2 = 6;                  // e4m3: a tile's largest row is scaled to codes of 64 times their value
constexpr float kLift = 64.0f;
constexpr float kKeyBound = 0.0079f;          // of what a key's factor leaves of its scale, from 1: a little above 2^-7
constexpr float kBoundedScore = 100.0f;       // largest score that the bound is used for
// Query rows whose largest element lies in [2^-6, 2^10) are lifted by 2^5: elements down to 2^-16 of the row's largest stay exact
// in f16, and the others are off by 2^-24 of it at most. Other rows have a power of their own.
constexpr float kCommonLift = 32.0f, kCommonLeast = 0x1p-6f, kCommonMost = 0x1p10f;

template <int HD, bool E4M3>
struct TilesCfg {
  static constexpr int kHalves = HD / 64;
  static constexpr int kTile = kHalves * kHalf;
  static constexpr int kRing = E4M3 ? 3 : (HD == 128 ? 4 : 6);     // 16-bit key / value tiles
  static constexpr int kCodes = kKeys * HD;                        // e4m3 bytes of a tile
  static constexpr int kStages = HD == 128 ? 3 : 6;                // tiles of codes on their way
  static constexpr int kSegs = HD / 16;                            // 16-byte segments of a row of codes
  static constexpr int kScaleBufs = 4;
  // registers of a softmax thread and of the others: together those of two threads at launch
  static constexpr int kSoftmaxRegs = E4M3 ? 136 : 152, kOtherRegs = 256 - kSoftmaxRegs;
  static constexpr int kQ = 0;
  static constexpr int kRingOff = 2 * kTile;
  static constexpr int kCodeOff = kRingOff + kRing * kTile;
  static constexpr int kRawScaleOff = kCodeOff + (E4M3 ? kStages * kCodes : 0);  // scales on their way: [kStages][2][128]
  static constexpr int kScaleOff = kRawScaleOff + (E4M3 ? kStages * 2 * kKeys * 4 : 0);   // float4 of each scale buffer
  static constexpr int kKeyOff = kScaleOff + (E4M3 ? kScaleBufs * 16 : 0);                 // [kScaleBufs][128] keys' words
  static constexpr int kFactorOff = kKeyOff + (E4M3 ? kScaleBufs * kKeys * 4 : 0);         // [2][128] half2, [8] maxima
  static constexpr int kBarOff = kFactorOff + (E4M3 ? 2 * kKeys * 4 + 32 : 0);
  static constexpr int kQScaleOff = kBarOff + 512;                 // e4m3: [2][tile][128] scales of the query rows
  static constexpr int kWalkOff = kQScaleOff + (E4M3 ? 2 * 2 * 128 * 4 : 0);
  static constexpr int kBytes = kWalkOff + 16 * 64 + 1024;
};

// tcgen05.mma with A from TMEM.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// True in one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
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
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { ptx::tmem_ld_32x32b_x32(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) { tmem_st_x32(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
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
__device__ __forceinline__ uint64_t pair_u(uint32_t x, uint32_t y) { return pair(__uint_as_float(x), __uint_as_float(y)); }

// One step (BIT 1, then 2) of a turn within four lanes: from a row of four 32-byte pieces in each lane to piece k of row
// k ... of all four rows in lane k, piece after piece. Stored as they come out of TMEM, a row to a thread, a warp's 32 pieces
// lie in 32 lines, which the load/store unit takes one by one: an item's output kept it busy for 5000 cycles of the 9000 that
// an item of one tile took. Turned, four lanes write a whole line.
template <int BIT>
__device__ __forceinline__ void turn4(uint32_t (&z)[32], int lane) {
  const bool odd = (lane & BIT) != 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s & BIT) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t &lo = z[8 * s + e], &hi = z[8 * (s | BIT) + e];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, BIT);
      (odd ? lo : hi) = got;
    }
  }
}
// A key's word is the factor of its scores; its last byte says what is left of its value's scale: here -(2 + byte 2^-14), so
// that P (1 + byte 2^-14) is -(P + P times it).
__device__ __forceinline__ float value_rest(float word) { return __uint_as_float(__byte_perm(__float_as_uint(word), 0xc0000000u, 0x7504)); }
// Barrier of the four warps that turn codes into f16.
__device__ __forceinline__ void converters_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Eight e4m3 codes as f16, times a factor.
__device__ __forceinline__ uint4 scaled(uint32_t x, uint32_t y, __half2 f) {
  uint32_t h[4];
  e4m3x4_f16x4(x, h[0], h[1]);
  e4m3x4_f16x4(y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), f);
    h[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}
// 3-D tiled load; c0 is the innermost coordinate.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Untiled bulk copy (both addresses and the size multiples of 16 bytes).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, int bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(ptx::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
               : "memory");
}

// Where a warp is in the CTA's list of work: each role walks on its own.
struct alignas(64) Walk {
  TileWork it;
  int at, last;
};

template <int HD, bool E4M3>
__global__ void __launch_bounds__(kThreads, 1)
attention_tiles_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ CUtensorMap tmap_q, uint16_t* __restrict__ o, float scale_log2, float scale_power, KvView kv,
                       SeqView v) {
  using C = TilesCfg<HD, E4M3>;
  constexpr int kSteps = HD / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_u32(smem);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* kv_empty = kv_full + C::kRing;
  uint64_t* q_full = kv_empty + C::kRing;
  uint64_t* q_empty = q_full + 2;
  uint64_t* q_raw = q_empty + 2;                      // e4m3: bf16 queries that are not f16 yet
  uint64_t* s_full = q_raw + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* sc_full = o_full + 2;                     // [kScaleBufs]
  uint64_t* v_short = sc_full + C::kScaleBufs;        // bf16: a value tile with rows past the length is there, and
  uint64_t* v_clean = v_short + 1;                    // those rows are zero
  uint64_t* raw_full = v_clean + 1;                   // [kStages], e4m3
  uint64_t* raw_empty = raw_full + C::kStages;
  uint64_t* drained = raw_empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  float* q_scale = reinterpret_cast<float*>(smem + C::kQScaleOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* err = v.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRing; ++i) {
      ptx::mbar_init(&kv_full[i], E4M3 ? 128 : 1);
      ptx::mbar_init(&kv_empty[i], 1);
    }
    for (int w = 0; w < 2; ++w) {
      ptx::mbar_init(&q_full[w], E4M3 ? 32 : 1);
      ptx::mbar_init(&q_raw[w], 1);
      ptx::mbar_init(&q_empty[w], 1);
      ptx::mbar_init(&s_full[w], 1);
      ptx::mbar_init(&p_full[w], 128);
      ptx::mbar_init(&o_full[w], 1);
    }
    for (int i = 0; i < C::kScaleBufs; ++i) ptx::mbar_init(&sc_full[i], 128);
    ptx::mbar_init(v_short, 1);
    ptx::mbar_init(drained, 1);
    ptx::mbar_init(v_clean, 32);
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(&raw_full[i], 1);
      ptx::mbar_init(&raw_empty[i], 128);
    }
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

  // Each warp's walk lives in shared memory: the fields are read a few times an item, and a softmax thread has no
  // registers to keep them in.
  Walk& walk = reinterpret_cast<Walk*>(smem + C::kWalkOff)[warp];      // [16]
  const TileWork& it = walk.it;
  auto load = [&](int at) {
    constexpr int kWords = sizeof(TileWork) / 4;
    const int x = lane < kWords ? reinterpret_cast<const int*>(v.tile_work + at)[lane] : at;
    __syncwarp();
    if (lane <= kWords) reinterpret_cast<int*>(&walk)[lane] = x;
    __syncwarp();
  };
  bool any;
  {
    const int2 share = v.tile_share[blockIdx.x];
    any = share.y > 0;
    if (any) load(share.x);
    if (lane == 0) walk.last = share.x + share.y - 1;
    __syncwarp();
  }
  auto advance = [&]() {
    __syncwarp();
    const int at = walk.at;
    if (at == walk.last) return false;
    load(at + 1);
    return true;
  };
  bool dead = false;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead && !ptx::mbar_wait(bar, parity, err)) dead = true;
  };

  // Keys and values of the share's tiles into the ring (bf16), or codes and scales into the stages (e4m3): one warp, a
  // lane for each page of a tile.
  auto bring = [&]() {
    uint64_t* full = E4M3 ? raw_full : kv_full;
    uint64_t* empty = E4M3 ? raw_empty : kv_empty;
    constexpr int kDepth = E4M3 ? C::kStages : C::kRing;
    const int box = min(kv.page, kKeys), boxes = kKeys / box;
    uint32_t n = 0;                                   // tiles brought so far
    for (bool go = any; go; go = advance()) {
      const int32_t* table = v.table + static_cast<size_t>(it.seq) * v.max_pages;
      for (int j = it.ka; j < it.kb; ++j) {
        const int key = j * kKeys + lane * box;
        const bool mine = lane < boxes && key < it.len;
        int at = 0;
        if (mine) at = ((table[key >> kv.page_log2] * v.Hkv + it.kvh) << kv.page_log2) + (key & (kv.page - 1));
        const int count = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll
        for (int h = 0; h < 2; ++h, ++n) {            // the keys (and both scales), then the values
          const int st = n % kDepth;
          wait(&empty[st], ((n / kDepth) & 1) ^ 1);
          if (__any_sync(0xffffffffu, dead)) return;
          if (lane == 0)
            ptx::mbar_arrive_expect_tx(&full[st], count * box * (!E4M3 ? 2 * HD : h == 0 ? HD + 8 : HD));
          __syncwarp();
          if (!mine) continue;
          if (E4M3) {
            ptx::tma_load_2d(smem + C::kCodeOff + st * C::kCodes + lane * box * HD, h ? &tmap_v : &tmap_k, &full[st], 0, at);
            if (h == 0) {
              uint8_t* dst = smem + C::kRawScaleOff + st * 2 * kKeys * 4 + lane * box * 4;
              bulk_load(dst, kv.k_scale + at, box * 4, &full[st]);
              bulk_load(dst + kKeys * 4, kv.v_scale + at, box * 4, &full[st]);
            }
          } else {
            uint8_t* dst = smem + C::kRingOff + st * C::kTile + lane * box * 128;
#pragma unroll
            for (int x = 0; x < C::kHalves; ++x)
              ptx::tma_load_2d(dst + x * kHalf, h ? &tmap_v : &tmap_k, &full[st], 64 * x, at);
          }
        }
      }
    }
  };

  if (warp < 8) {
    // ------------------------------------------------------------------ softmax of tile w
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int w = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128 * w, to = tmem + lanes + 256 + 128 * w;
    const bool wide = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
    const int row_tok = row / v.G, row_head = row - row_tok * v.G;
    uint32_t n_s = 0, n_o = 0;                        // waits done on s_full, o_full
    uint32_t n_sc = 0;                                // key tiles of the CTA so far (scale buffers)
    for (bool go = any; go;) {
      const int tok = it.t0 + v.tile_tokens * w + row_tok;
      const bool valid = row_tok < v.tile_tokens && tok < it.n;
      const int lim = valid ? it.len - it.n + tok : -1;
      // the fewest and the most keys that a row of the warp sees (rows of no token see none)
      const int low = __reduce_min_sync(0xffffffffu, valid ? lim : INT_MAX), high = __reduce_max_sync(0xffffffffu, lim);
      const int ka = it.ka, end = it.end[w];
      float c = scale_log2;                           // e4m3: the query row's power of two beside the common one
      bool plain = true;                              // e4m3: 1 in all rows of the warp
      float m = -INFINITY, l = 0.f;
      for (int j = ka; j < end; ++j) {
        // score = S c + off; e4m3: S c key[column] + off, key[] near cs; the sum takes rv times the exponentials
        float off = 0.f, rv = 1.f, cs = 1.f;
        const float* key = nullptr;
        wait(&s_full[w], n_s & 1);
        ++n_s;
        ptx::tc_fence_after();
        if (E4M3) {
          // (The query rows' scales were there before the products that s_full stands for. So were the tile's factors, and
          // they are not waited for any sooner: a tile without work in an item comes here while the codes of that item are
          // still on their way, when the factors' barrier may be two phases back, which its parity cannot tell.)
          const uint32_t t = n_sc + (j - ka);
          wait(&sc_full[t % C::kScaleBufs], (t / C::kScaleBufs) & 1);
          const float4 f = reinterpret_cast<const float4*>(smem + C::kScaleOff)[t % C::kScaleBufs];
          cs = f.x, off = f.y, rv = f.z;
          key = reinterpret_cast<const float*>(smem + C::kKeyOff) + (t % C::kScaleBufs) * kKeys;
          if (j == ka) {
            c = valid ? q_scale[((n_o & 1) * 2 + w) * 128 + row] * scale_power : 1.f;
            plain = __all_sync(0xffffffffu, c == 1.f);
          }
        }
        const uint64_t cc = pair(c, c);
        const int seen = lim - j * kKeys, seen_low = low - j * kKeys, seen_high = high - j * kKeys;   // keys 0 .. seen are visible
        constexpr int W = 32;                         // columns at a time
        auto mask = [&](uint32_t (&x)[W], int h) {    // of columns W h ...
#pragma unroll
          for (int i = 0; i < W; ++i) x[i] = W * h + i > seen ? 0xff800000u : x[i];
        };
        const bool edge = seen_low < kKeys - 1;       // some row of the warp does not see the whole tile
        auto largest = [&](const uint32_t (&x)[W], float t) {
          float u = __uint_as_float(x[0]);
#pragma unroll
          for (int i = 1; i < W / 2; ++i) {
            u = fmaxf(u, __uint_as_float(x[i]));
            t = fmaxf(t, __uint_as_float(x[i + W / 2]));
          }
          return fmaxf(fmaxf(t, __uint_as_float(x[W / 2])), u);
        };
        uint32_t xa[W], xb[W];
        float top = -INFINITY;
        uint64_t sum = 0, sum1 = 0;                   // two zeros each
        auto rescale = [&](float next) {
          const float f = next == m ? 1.f : exp2_approx(m - next);
          m = next;
          l *= f;
#pragma unroll 1
          for (int i = 0; i < HD / W; ++i) {
            tmem_ld(to + W * i, xb);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < W; ++k) xb[k] = __float_as_uint(__uint_as_float(xb[k]) * f);
            tmem_st(to + W * i, xb);
          }
        };
        // the weights of columns W h ... against the maximum m, into p; e4m3: kf: the columns' words
        auto weights = [&](uint32_t (&x)[W], uint64_t neg, uint32_t* p, const float4* kf) {
#pragma unroll
          for (int i = 0; i < W; i += 4) {
            const uint64_t c0 = E4M3 ? pair(kf[i / 4].x, kf[i / 4].y) : cc, c1 = E4M3 ? pair(kf[i / 4].z, kf[i / 4].w) : cc;
            float2 e0 = unpair(fma_pair(pair_u(x[i], x[i + 1]), c0, neg));
            float2 e1 = unpair(fma_pair(pair_u(x[i + 2], x[i + 3]), c1, neg));
            e0.x = exp2_approx(e0.x), e0.y = exp2_approx(e0.y);
            e1.x = exp2_approx(e1.x), e1.y = exp2_approx(e1.y);
            const uint64_t y0 = pair(e0.x, e0.y), y1 = pair(e1.x, e1.y);
            sum = add_pair(sum, y0);
            sum1 = add_pair(sum1, y1);
            if (E4M3) {                               // -P: the value rows are negative too
              e0 = unpair(fma_pair(y0, pair(value_rest(kf[i / 4].x), value_rest(kf[i / 4].y)), y0));
              e1 = unpair(fma_pair(y1, pair(value_rest(kf[i / 4].z), value_rest(kf[i / 4].w)), y1));
            }
            p[i / 2] = E4M3 ? pack_f16(e0.x, e0.y) : pack_bf16(e0.x, e0.y);
            p[i / 2 + 1] = E4M3 ? pack_f16(e1.x, e1.y) : pack_bf16(e1.x, e1.y);
          }
        };
        if (E4M3 || edge) {
          // Two passes over S in small loops: the maximum, then the weights, each piece's P over columns of S that were
          // read. e4m3: the supply of instructions bounds it, since converters and softmax run different code side by side;
          // held as below, unrolled, the warps waited for instructions more often than they issued one (8000 tokens 621 us
          // against 568; two pieces a turn, the next loaded ahead, 625). bf16: for the tiles that some row of the warp
          // does not see whole, at most two of an item, where a second unrolled copy cost registers (347 us against 335).
          const int pieces = max(0, min(kKeys / W, (seen_high + W) / W));         // that some row of the warp sees
          auto load_keys = [&](float4 (&f)[W / 4], int h) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) f[i] = reinterpret_cast<const float4*>(key + W * h)[i];
          };
          auto maximum = [&](auto exact) {            // of S, or of S times the keys' factors
            float t = -INFINITY;
#pragma unroll 1
            for (int h = 0; h < pieces; ++h) {
              tmem_ld(ts + W * h, xa);
              ptx::tmem_ld_wait();
              if (exact.value) {
                float4 f[W / 4];
                load_keys(f, h);
#pragma unroll
                for (int i = 0; i < W; ++i) xa[i] = __float_as_uint(__uint_as_float(xa[i]) * (&f[i / 4].x)[i & 3]);
              }
              if (edge) mask(xa, h);
              t = largest(xa, t);
            }
            return t;
          };
          top = maximum(std::false_type{}) * (E4M3 ? c * cs : c);
          if (E4M3) {
            const bool far = fabsf(top) > kBoundedScore && top != -INFINITY;
            top = fmaf(kKeyBound, fminf(fabsf(top), kBoundedScore), top) + off;
            if (__any_sync(0xffffffffu, far)) {       // (for those rows alone: a row's result is its own)
              const float exact = fmaf(maximum(std::true_type{}), c, off);
              top = far ? exact : top;
            }
          }
          if (j == ka)
            m = top;
          else if (__any_sync(0xffffffffu, top > m + kLazy<E4M3>))
            rescale(top > m + kLazy<E4M3> ? top : m);
          const float mm = m == -INFINITY ? 0.f : m;
          const uint64_t neg = pair(off - mm + kUp<E4M3>, off - mm + kUp<E4M3>);
          uint32_t p[W / 2];
          auto second = [&](auto scaled) {
#pragma unroll 1
            for (int h = 0; h < pieces; ++h) {
              float4 f[W / 4];
              tmem_ld(ts + W * h, xa);
              if (E4M3) load_keys(f, h);              // (on their way together)
              ptx::tmem_ld_wait();
              if (scaled.value) {
#pragma unroll
                for (int i = 0; i < W; ++i) xa[i] = __float_as_uint(__uint_as_float(xa[i]) * c);
              }
              if (edge) mask(xa, h);
              weights(xa, neg, p, f);
              tmem_st(ts + W / 2 * h, p);
            }
          };
          if (!E4M3 || plain)
            second(std::false_type{});
          else
            second(std::bool_constant<E4M3>{});
          if (pieces < kKeys / W) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) p[i] = 0u;
#pragma unroll 1
            for (int h = max(pieces, 0); h < kKeys / W; ++h) tmem_st(ts + W / 2 * h, p);
          }
        } else {
          if (j == ka) {                              // a first maximum: that of the first columns
            tmem_ld(ts, xa);
            ptx::tmem_ld_wait();
            m = fmaf(largest(xa, top), c, off);
          }
          // One pass over S, W columns at a time: weights against the maximum so far, and the tile's own maximum. P
          // waits in registers: where the tile's maximum is above the lazy limit, S is still there for another pass.
          uint32_t p[64];
          for (;;) {
            const float mm = m == -INFINITY ? 0.f : m;
            const uint64_t neg = pair(off - mm, off - mm);
            top = -INFINITY;
            sum = 0, sum1 = 0;
            auto piece = [&](uint32_t (&x)[W], int h) {
              top = largest(x, top);
              weights(x, neg, p + W / 2 * h, nullptr);
            };
            tmem_ld(ts, xa);
#pragma unroll
            for (int h = 0; h < kKeys / W; h += 2) {
              ptx::tmem_ld_wait();
              tmem_ld(ts + W * h + W, xb);
              piece(xa, h);
              ptx::tmem_ld_wait();
              if (h + 2 < kKeys / W) tmem_ld(ts + W * h + 2 * W, xa);
              piece(xb, h + 1);
            }
            top = fmaf(top, c, off);
            if (!__any_sync(0xffffffffu, top > m + kLazy<E4M3>)) break;
            rescale(top > m + kLazy<E4M3> ? top : m);
          }
          tmem_st_x32(ts, p);
          tmem_st_x32(ts + 32, p + 32);
        }
        const float2 total = unpair(add_pair(sum, sum1));
        l = fmaf(total.x + total.y, rv, l);
        tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&p_full[w]);
      }
      n_sc += it.kb - ka;
      // While the last product runs: where the rows go, and the next item.
      const bool part = it.split != 0 && it.t0 + v.tile_tokens * w < it.n;     // of a split item, to the workspace
      const float inv = inverse(l);
      const int64_t own = (static_cast<int64_t>(it.start + tok) * v.Hq + it.kvh * v.G + row_head) * HD;
      uint16_t* dst[4];                               // of the rows of the thread's four lanes, where the thread stores
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t of = __shfl_sync(0xffffffffu, valid ? own : -1, (lane & ~3) + k);
        dst[k] = of < 0 ? nullptr : o + of + 16 * (lane & 3);
      }
      float* mine = v.tile_part + ((2 * static_cast<int64_t>(blockIdx.x) + (ka == 0)) * 2 + w) * tile_slot(v);
      const bool worked = end > ka;
      go = advance();
      if (worked) {
        wait(&o_full[w], n_o & 1);
        ++n_o;
        ptx::tc_fence_after();
      }
      if (part) {
        if (worked) {
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
      } else if (worked) {
        uint32_t y0[32], y1[32];
        tmem_ld(to, y0);
        tmem_ld(to + 32, y1);
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
          uint32_t z[32];
          ptx::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            z[k] = pack_bf16(__uint_as_float(y0[2 * k]) * inv, __uint_as_float(y0[2 * k + 1]) * inv);
            z[16 + k] = pack_bf16(__uint_as_float(y1[2 * k]) * inv, __uint_as_float(y1[2 * k + 1]) * inv);
          }
          if (i + 1 < HD / 64) {
            tmem_ld(to + 64, y0);
            tmem_ld(to + 96, y1);
          }
          turn4<1>(z, lane);
          turn4<2>(z, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (dst[k] != nullptr) store32(dst[k] + 64 * i, z + 8 * k, wide);
        }
      }
      ptx::tc_fence_before();
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------------ keys and values
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (!E4M3) {
      if (warp == 8) {
        bring();
      } else if (warp == 9) {
        // value rows past the length, in the one tile of an item that may hold any, when the products have come to it
        uint32_t n = 1, par = 0;                      // ring position of the item's first value tile; tiles so far
        for (bool go = any; go; go = advance()) {
          if (it.kb * kKeys > it.len) {
            wait(v_short, par);
            par ^= 1;
            uint8_t* t = smem + C::kRingOff + (n + 2 * (it.kb - 1 - it.ka)) % C::kRing * C::kTile;
            for (int i = (it.len - (it.kb - 1) * kKeys) * (HD / 8) + lane; i < kKeys * (HD / 8); i += 32)
              *reinterpret_cast<uint4*>(t + (i % (HD / 8) >> 3) * kHalf + i / (HD / 8) * 128 + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(v_clean);
          }
          n += 2 * (it.kb - it.ka);
        }
      }
    } else {
      const int tid = threadIdx.x - 256;
      constexpr int kStep = 128 / C::kSegs;           // rows that the threads take at a time, 16 codes each
      constexpr int kCopies = kKeys / kStep;
      const int seg = tid % C::kSegs, r_in = tid / C::kSegs, even = (seg & 3) * 2;
      const bool odd = seg >= 4;                      // the second half tile's lanes take their two segments in the
                                                      // other order: different banks
      __half2* factors = reinterpret_cast<__half2*>(smem + C::kFactorOff);           // keys' rows, values' rows
      float* maxima = reinterpret_cast<float*>(smem + C::kFactorOff + 2 * kKeys * 4);
      uint32_t n = 0;
      for (bool go = any; go; go = advance()) {
        for (int j = it.ka; j < it.kb; ++j) {
          const int cut = it.len - j * kKeys;         // rows of the tile inside the sequence (any number)
#pragma unroll 1
          for (int h = 0; h < 2; ++h, ++n) {
            const int st = n % C::kRing, cs = n % C::kStages;
            wait(&raw_full[cs], (n / C::kStages) & 1);
            if (h == 0) {
              // the tile's largest scales, and every row's share of them. A row with a NaN scale is NaN in its
              // scores alone: its values would reach rows that do not see it.
              const float* rw = reinterpret_cast<const float*>(smem + C::kRawScaleOff) + cs * 2 * kKeys + tid;
              float ks = tid < cut ? rw[0] : 0.f, vs = tid < cut ? rw[kKeys] : 0.f;
              const bool none = !(fabsf(ks) < kMostScale) || !(fabsf(vs) < kMostScale);
              if (none) ks = vs = 0.f;
              float km = fabsf(ks), vm = vs;
#pragma unroll
              for (int d = 16; d > 0; d >>= 1) {
                km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, d));
                vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, d));
              }
              if (lane == 0) maxima[warp - 8] = km, maxima[warp - 4] = vm;
              converters_sync();
              km = fmaxf(fmaxf(maxima[0], maxima[1]), fmaxf(maxima[2], maxima[3]));
              vm = fmaxf(fmaxf(maxima[4], maxima[5]), fmaxf(maxima[6], maxima[7]));
              if (!(km >= kLeastScale)) km = 1.f;
              if (!(vm >= kLeastScale)) vm = 1.f;
              const uint32_t kp = __float_as_uint(km) & 0x7f800000, vp = __float_as_uint(vm) & 0x7f800000;   // the powers below
              const float ki = __uint_as_float((254u << 23) - kp), vi = __uint_as_float((254u << 23) - vp);   // their inverses
              const uint32_t t = n / 2;
              // the scales to 7 bits, the key's to the nearest, as shares of those powers; what is left of the value's scale,
              // 1 + byte 2^-14, lies in the last bits of what is left of the key's
              const float k7 = __int_as_float((__float_as_int(ks) + 0x10000) & 0xfffe0000);
              const float v7 = vs >= kLeastScale ? __int_as_float(__float_as_int(vs) & 0xfffe0000) : 0.f;
              factors[tid] = __half2half2(__float2half_rn(none ? __int_as_float(0x7fffffff) : kLift * (k7 * ki)));
              factors[kKeys + tid] = __half2half2(__float2half_rn(-kLift * (v7 * vi)));
              const float common = scale_log2 * (__uint_as_float(kp) * (1.0f / (kLift * kCommonLift)));
              const int key = __float_as_int(fabsf(ks) >= kLeastScale ? common * __fdividef(ks, k7) : common);
              const int byte = v7 > 0.f ? min(255, __float2int_rn(__fdividef(vs - v7, v7) * 16384.f)) : 0;
              (reinterpret_cast<int*>(smem + C::kKeyOff) + (t % C::kScaleBufs) * kKeys)[tid] = ((key - byte + 128) & ~255) | byte;
              if (tid == 0)
                reinterpret_cast<float4*>(smem + C::kScaleOff)[t % C::kScaleBufs] =
                    make_float4(common, static_cast<float>((__float_as_int(vm) >> 23) - 127 - kLiftLog2), vi * kLift, 0.f);
              ptx::mbar_arrive(&sc_full[t % C::kScaleBufs]);
              converters_sync();
            }
            wait(&kv_empty[st], ((n / C::kRing) & 1) ^ 1);
            const uint8_t* src = smem + C::kCodeOff + tid * 16 + cs * C::kCodes;
            uint8_t* dst = smem + C::kRingOff + st * C::kTile + (seg >> 2) * kHalf;
            constexpr int kAtOnce = 4;                // (2: 597 us at 8000 tokens, 8 the same as 4)
#pragma unroll 1
            for (int i0 = 0; i0 < kCopies; i0 += kAtOnce) {
              uint2 cd[kAtOnce][2];
              __half2 f[kAtOnce];
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  cd[i][x] = *reinterpret_cast<const uint2*>(src + (i0 + i) * 2048 + (x ^ (odd ? 1 : 0)) * 8);
                f[i] = factors[h * kKeys + (i0 + i) * kStep + r_in];
              }
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
                const int r = (i0 + i) * kStep + r_in;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  uint4 y = scaled(cd[i][x].x, cd[i][x].y, f[i]);
                  if (r >= cut) y = make_uint4(0u, 0u, 0u, 0u);
                  *reinterpret_cast<uint4*>(dst + r * 128 + (((even + (x ^ (odd ? 1 : 0))) ^ (r & 7)) * 16)) = y;
                }
              }
            }
            ptx::mbar_arrive(&raw_empty[cs]);
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&kv_full[st]);
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == 12) {
      // ---------------------------------------------------------------- products
      if (elect_one()) {
        const uint32_t id_s = idesc16(E4M3, 128, kKeys, false), id_o = idesc16(E4M3, 128, HD, true);
        uint32_t ks = 0, ks_par = 0, vs = 0, vs_par = 0;           // ring slots of K_j and V_{j-1}, their phases
        uint32_t q_par[2] = {0, 0}, p_par[2] = {0, 0}, clean_par = 0;
        int at = any ? walk.at : 0, len = it.len;
        const int last = any ? walk.last : -1;
        int4 next = *reinterpret_cast<const int4*>(&it);
        while (at <= last) {
          const int ka = next.x, kb = next.y, end0 = next.z, end1 = next.w;
          const bool short_tile = !E4M3 && kb * kKeys > len;
          if (++at <= last) {                         // the next item, long before it is wanted
            next = *reinterpret_cast<const int4*>(v.tile_work + at);
            len = v.tile_work[at].len;
          }
          for (int j = ka; j <= kb; ++j) {
            if (j > ka) {
              vs = ks, vs_par = ks_par;               // the tile after K_{j-1}
              if (++vs == C::kRing) vs = 0, vs_par ^= 1;
              ks = vs, ks_par = vs_par;
              if (++ks == C::kRing) ks = 0, ks_par ^= 1;
              wait(&kv_full[vs], vs_par);
              if (dead) break;
              if (short_tile && j == kb) {
                ptx::mbar_arrive(v_short);
                wait(v_clean, clean_par);
                clean_par ^= 1;
              }
            }
            if (j < kb) wait(&kv_full[ks], ks_par);
            const uint64_t dv = kDescN + ((base + C::kRingOff + vs * C::kTile) >> 4);
            const uint64_t dk = kDescK + ((base + C::kRingOff + ks * C::kTile) >> 4);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int end = w ? end1 : end0;
              if (j > ka && j - 1 < end) {
                wait(&p_full[w], p_par[w]);
                p_par[w] ^= 1;
                ptx::tc_fence_after();
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  umma_ts(tmem + 256 + 128 * w, tmem + 128 * w + 8 * k, dv + k * (2048 >> 4), id_o, j - 1 > ka || k > 0);
                if (j == end) ptx::umma_commit(&o_full[w]);
              }
              if (j < end) {
                if (j == ka) {
                  wait(&q_full[w], q_par[w]);
                  q_par[w] ^= 1;
                  ptx::tc_fence_after();
                }
                const uint64_t dq = kDescK + ((base + C::kQ + w * C::kTile) >> 4);
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                  const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
                  ptx::umma_bf16(tmem + 128 * w, dq + off, dk + off, id_s, k > 0);
                }
                ptx::umma_commit(&s_full[w]);
                if (j + 1 == end) ptx::umma_commit(&q_empty[w]);
              }
            }
            if (j > ka) ptx::umma_commit(&kv_empty[vs]);
            if (j < kb) ptx::umma_commit(&kv_empty[ks]);
          }
          if (dead) break;
          // (ks is now the slot of the next item's first key tile)
        }
        if (dead) {                                   // the products under way
          ptx::umma_commit(drained);
          ptx::mbar_wait(drained, 0, err);
        }
      }
      __syncwarp();
    } else if (warp == 14) {
      if (E4M3) bring();
    } else {
      // ---------------------------------------------------------------- queries
      // TMA boxes of whole tokens (rows past the tile's last token keep what was there, rows of other sequences may come
      // along: their results are not used)
      const int w = warp == 13;
      uint32_t par = 0;
      const uint32_t bytes = static_cast<uint32_t>(v.tile_tokens * v.G * HD * 2);
      uint8_t* tile = smem + C::kQ + w * C::kTile;
      uint64_t* full = E4M3 ? &q_raw[w] : &q_full[w];
      for (bool go = any; go; go = advance()) {
          if (it.end[w] <= it.ka) continue;
        wait(&q_empty[w], par ^ 1);
        if (__any_sync(0xffffffffu, dead)) break;
        if (lane == 0) {
          ptx::mbar_arrive_expect_tx(full, bytes);
#pragma unroll
          for (int x = 0; x < C::kHalves; ++x)
            tma_load_3d(tile + x * kHalf, &tmap_q, full, 64 * x, it.kvh * v.G, it.start + it.t0 + v.tile_tokens * w);
        }
        __syncwarp();
        if (E4M3) {
          // to f16, each row lifted by a power of two: two lanes to a row
          constexpr int kN = HD / 16;                 // a lane's 16-byte segments
          wait(full, par);
#pragma unroll 1
          for (int r0 = 0; r0 < 128; r0 += 16) {
            const int row = r0 + (lane >> 1), side = lane & 1;
            uint4 x[kN];
            float most = 0.f;
            auto seg = [&](int i) { return reinterpret_cast<uint4*>(tile + ((i + side * kN) >> 3) * kHalf + row * 128 + ((((i + side * kN) & 7) ^ (row & 7)) * 16)); };
#pragma unroll
            for (int i = 0; i < kN; ++i) x[i] = *seg(i);
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              const uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) most = fmaxf(most, fmaxf(fabsf(ptx::bf16_lo(y[k])), fabsf(ptx::bf16_hi(y[k]))));
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            float back, lift = query_lift(most, &back);
            if (most == 0.f || (most >= kCommonLeast && most < kCommonMost)) lift = kCommonLift, back = 1.0f / kCommonLift;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
              uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = pack_f16(ptx::bf16_lo(y[k]) * lift, ptx::bf16_hi(y[k]) * lift);
              *seg(i) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            if (side == 0) q_scale[(par * 2 + w) * 128 + row] = back * kCommonLift;
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(&q_full[w]);
        }
        par ^= 1;
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
  CUtensorMap tq;
  if (!make_tmap_heads_bf16(&tq, q, s.T, s.Hq, HD, s.tile_tokens, s.G)) return cudaErrorInvalidValue;
  using C = TilesCfg<HD, E4M3>;
  if (cudaError_t e = allow_shared_memory<attention_tiles_kernel<HD, E4M3>>(C::kBytes)) return e;
  // e4m3: an unusual scale's power of two goes with the query rows, so that the keys' factors are normal numbers
  float power = 1.0f;
  if (E4M3 && !(scale_log2 > 0x1p-16f && scale_log2 < 0x1p16f)) power = std::ldexp(1.0f, std::max(-126, std::ilogb(scale_log2)));
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attention_tiles_kernel<HD, E4M3>, tk, tv, tq, o, scale_log2 / power, power, kv, s);
  note_launch_end(kKindAttn, st);
  return e;
}

}  // namespace

bool make_kv_maps(const KvView& kv, CUtensorMap* k, CUtensorMap* v) {
  const long rows = static_cast<long>(kv.n_pages) * kv.page * kv.Hkv;
  const int box = std::min(kv.page, kTileKeys);
  if (kv.type == kKvE4m3) return make_tmap_u8(k, kv.K, rows, kv.hd, box) && make_tmap_u8(v, kv.V, rows, kv.hd, box);
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
