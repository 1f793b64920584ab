// Declarations shared by the attention step's translation units: device-side views of a paged
// KV cache and of one step's sequences, and the kernels' launchers. Not part of the C ABI.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace mlora {

constexpr int kKvBf16 = 0, kKvE4m3 = 1;

// The smallest magnitude a cached row's scale is made for: a row whose largest element is below
// it quantises against it, so that every scale is a normal fp32 number with a normal reciprocal.
constexpr float kAmaxMin = 8.673617379884035e-19f;   // 2^-60
constexpr float kE4m3Max = 448.0f;
// Scales below this count as zero, those from the other one on as NaN (those written here lie between 2^-69 and 2^120).
constexpr float kLeastScale = 0x1p-100f, kMostScale = 0x1p120f;

// Device arrays of one layer's paged cache. Row (page, head, offset) of K and V holds hd elements.
struct KvView {
  void* K;            // [n_pages, Hkv, page, hd] bf16 or e4m3
  void* V;            // the same
  float* k_scale;     // [n_pages, Hkv, page] fp32 (e4m3 caches only)
  float* v_scale;
  int n_pages, page, page_log2, Hkv, hd, type;
};

// A sequence of the row kernel's list, and a CTA's share of the list: `units` units of 64 keys, from unit `unit` of head
// kvh of list entry `item` on.
struct RowSeq {
  int32_t seq, n, len, start;
};
// Where the share begins (ends) inside an item, first_cta (last_cta) is the CTA that has that item's first part, of
// first_parts (last_parts); otherwise the parts are 0.
struct alignas(16) RowShare {
  int32_t item, kvh, unit, units;
  int32_t first_cta, first_parts, last_cta, last_parts;
};
// A block of the tile kernel's list: tokens t0 ... (two tiles of SeqView::tile_tokens) of sequence seq, `tiles` key
// tiles.
struct alignas(32) TileBlk {
  int32_t seq, n, len, start, t0, tiles, gap;
};
// What a CTA of the tile kernel does next: key tiles [ka, kb) of head kvh of such a block, of which its tile w sees
// [ka, end[w]); split: not the whole item; gap: as below, or, in a prefix pass, the block's number. A CTA's list begins at
// tile_share.x and holds tile_share.y of them.
struct alignas(16) TileWork {
  int32_t ka, kb, end[2];
  int32_t len, n, start, t0;
  int32_t seq, kvh, split, gap;
};
// An item (list entry, head) that lies across cuts: CTAs cta ... cta + parts - 1 each hold a part.
struct JoinTask {
  int32_t item, kvh, cta, parts;
};

// Which keys the rows of a step's sequences see, as the kernels are compiled for it:
//   kSeeAll     a row at position p all keys up to p;
//   kSeeRanges  with a window, keys j <= p with j < sinks or j > p - window; behind a shared prefix, keys up to p from the end of
//               the prefix on, the rows' sums over the prefix's keys joined from SeqView::pre_part. The chunks (key tiles) of a
//               sequence that some row sees are counted without the gap between the first ones and the window (or without
//               the prefix): chunk c is chunk c + gap of the cache from gap_chunk on (key tile: from gap_tile on);
//   kSeePrefix  the pass over the shared prefixes: a "sequence" is a group, every row of it sees all `len` keys, a multiple
//               of kTileKeys, and its sums go to pre_part.
constexpr int kSeeAll = 0, kSeeRanges = 1, kSeePrefix = 2;

// Device arrays of one step's sequences, written by launch_build_seq.
struct SeqView {
  int32_t* start;       // [S] first token row of each sequence
  int32_t* n;           // [S] new tokens
  int32_t* len;         // [S] cached length, the new tokens among it (0: the sequence is skipped)
  int32_t* table;       // [S, max_pages] page of each cached page index in use
  int32_t* tok_seq;     // [T] sequence of each token (-1: in none, or its sequence is skipped)
  int32_t* tok_pos;     // [T] position of each token
  int32_t* tok_row;     // [T] page * page size + offset of the token's cache row (-1: none)
  int32_t* page_pre;    // [S + 1] cached pages of the sequences before each
  RowSeq* row_seq;      // [S] the row kernel's sequences
  int64_t* row_pre;     // [S + 1] units (kRowHead and one for 64 keys, for each kv head) before each of them
  TileBlk* blk;         // [blocks] the tile kernel's blocks
  int64_t* blk_pre;     // [blocks + 1] units (kTileHead and the key tiles, for each kv head) before each of them
  RowShare* row_share;  // [row_ctas]
  int2* tile_share;     // [tile_ctas]
  TileWork* tile_work;  // [blocks * Hkv + tile_ctas]
  int32_t* row_there;   // [3][row_ctas] parts there of the first run of the item that a CTA begins, that item's runs there, parts
                        // there of a later run that the CTA begins (all 0 between calls)
  JoinTask* tile_join;  // [counts[2]] the tile kernel's split items
  int32_t* counts;      // [1] first rejected sequence (INT32_MAX if none), [2] split items
  uint32_t* err;        // device error word (ptx::kErr* bits)
  int32_t* row_gap;     // [S] kSeeRanges: gap of each of the row kernel's sequences, in chunks
  int32_t* skip;        // [S] keys of each sequence that its group's prefix pass takes (0: none)
  int32_t* group;       // [S] its group
  int2* pre_at;         // [S] first block of its group in the prefix pass (-1: none), its first token among the group's
  int32_t* rep;         // [S] prefix pass: a sequence that has the group's table
  int32_t* first_blk;   // [S] prefix pass: the group's first block
  float* pre_part;      // sums over the prefix of block b's rows: slot (b * Hkv + head) * 2 + tile, as tile_part's
  float* row_part;      // partial results of the row kernel's split items
  float* tile_part;     // of the tile kernel's
  int S, T, max_pages, Hq, Hkv, G, hd;
  int tile_tokens;      // tokens of one 128-row tile of the tile kernel (128 / G)
  int row_limit;        // rows (new tokens * G) up to which a sequence takes the row kernel
  int row_ctas, tile_ctas;
  int see;              // kSee*
  int window, sinks;    // kSeeRanges (without a window: INT_MAX, 0)
  int gap_chunk, gap_tile;
};

// What a step's rows see beside plain causal attention, for launch_build_seq: a window (0: none), or groups of sequences that
// share a prefix (device arrays; the prefix pass's own view).
struct SeqReuse {
  int window, sinks;
  const int32_t* group_start;   // [n_groups + 1]
  const int32_t* prefix_len;    // [n_groups]
  int n_groups;
  SeqView prefix;
};

// Keys of one unit of the row kernel (four warps x 16 keys) and of one tile of the tile kernel.
constexpr int kRowUnit = 64, kRowChunk = 16;
constexpr int kRowHead = 3;           // units that an item's fixed costs (queries, joining the warps' sums) are worth
constexpr int kRowShort = 48;         // units up to which an item is not cut into more parts than are joined in one go
constexpr int kTileKeys = 128;
constexpr int kTileSnap = 2;          // key tiles that a split costs at least (1 and 0: a prompt of 3000 tokens in shares 93, 97 us for 87)
constexpr int kTileDeal = 12;         // key tiles above the mean up to which whole items are dealt out (6: 6 chunks of 300 on 4000 137 us for 108)
constexpr int kTileHead = 3;          // key tiles that an item's fixed costs (queries, first products, output) are worth

// Sequences of a group from which on its prefix is attended once for all: for a few rows the tile kernel takes 1.5 us an SM for 128
// keys, 2.8 over e4m3, where the row kernel takes 1.45 and 0.8 us for each sequence.
__host__ __device__ constexpr int share_seqs(bool e4m3) { return e4m3 ? 4 : 2; }

// CTAs of the row kernel on an SM: by the row limit (16 rather than 8) and the cache's type.
__host__ __device__ constexpr int rows_ctas_per_sm(bool sixteen, bool e4m3) { return e4m3 && !sixteen ? 3 : 2; }

// Per-pair rotation frequencies in turns per position, each as a sum of three floats.
struct RopeView {
  const float4* freq;   // [rot / 2]
  int rot;              // rotated elements of a head (0: none)
  int interleaved;      // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  float mscale;         // factor on cos and sin
};

cudaError_t launch_build_seq(const int32_t* q_start, const int32_t* kv_len, const int32_t* pages, int table_ld,
                             const SeqView& s, int max_new, const KvView& kv, const SeqReuse& reuse, cudaStream_t st);
cudaError_t launch_qkv_write(const float* qkv, int64_t ld, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                             const RopeView& rope, const int32_t* positions, uint16_t* q, const KvView& kv,
                             const SeqView& s, int num_sms, cudaStream_t st);
cudaError_t launch_kv_read(const int32_t* row_start, int64_t rows, uint16_t* k, uint16_t* v, const KvView& kv,
                           const SeqView& s, int num_sms, cudaStream_t st);
// Attention in up to three launches, each a programmatic dependent of the one before: the row kernel (sequences of at
// most SeqView::row_limit rows, and the zero rows of tokens in no sequence), with `tiles` the tile kernel (the other
// sequences; tk and tv: the maps of the cache's K and V), and the join of the items that were split among CTAs. Where groups
// share prefixes, the tile kernel and the join run over those first (kSeePrefix; the first of a step's launches waits for the
// work before it as a whole).
cudaError_t launch_attention_rows(const uint16_t* q, uint16_t* o, float scale, const KvView& kv, const SeqView& s,
                                  cudaStream_t st);
cudaError_t launch_attention_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const uint16_t* q, uint16_t* o,
                                   float scale, const KvView& kv, const SeqView& s, cudaStream_t st);
cudaError_t launch_attention_join(uint16_t* o, const SeqView& s, cudaStream_t st);
// K and V as matrices [n_pages * Hkv * page, hd] in boxes of min(page, 128) rows x 64 columns (bf16, swizzled) or
// whole rows (e4m3).
bool make_kv_maps(const KvView& kv, CUtensorMap* k, CUtensorMap* v);
// Parts of split items: 2 c + 0 is the part that CTA c continues, 2 c + 1 the one that it begins.
// Row kernel: [rows][hd] sums, then [rows] (maximum, sum of weights), rows = row_limit.
// Tile kernel: two 128-row tiles, each [hd / 4][128] four sums, then [128] maxima and [128] sums of weights.
__host__ __device__ inline int64_t row_slot(const SeqView& s) { return static_cast<int64_t>(s.row_limit) * (s.hd + 2); }
__host__ __device__ inline int64_t tile_slot(const SeqView& s) { return static_cast<int64_t>(128) * (s.hd + 2); }
// The most blocks that n tokens of s sequences make in the tile kernel's list.
inline int64_t most_blocks(const SeqView& v, int64_t n, int64_t s) { return n / (2 * v.tile_tokens) + s; }
// Units of the row kernel over `len` keys without a gap of so many chunks.
__host__ __device__ inline int row_units(int len, int gap) {
  return ((len + kRowChunk - 1) / kRowChunk - gap + kRowUnit / kRowChunk - 1) / (kRowUnit / kRowChunk);
}
// The first key behind the sinks that the row at position p sees.
__host__ __device__ inline int first_seen(int p, int window) { return p - window + 1 > 0 ? p - window + 1 : 0; }
inline size_t row_part_bytes(const SeqView& s) { return static_cast<size_t>(s.row_ctas) * 2 * 16 * (s.hd + 2) * 4; }
inline size_t tile_part_bytes(const SeqView& s) { return static_cast<size_t>(s.tile_ctas) * 2 * 2 * tile_slot(s) * 4; }

}  // namespace mlora
