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

// Device arrays of one layer's paged cache. Row (page, head, offset) of K and V holds hd elements.
struct KvView {
  void* K;            // [n_pages, Hkv, page, hd] bf16 or e4m3
  void* V;            // the same
  float* k_scale;     // [n_pages, Hkv, page] fp32 (e4m3 caches only)
  float* v_scale;
  int n_pages, page, page_log2, Hkv, hd, type;
};

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
  int64_t* row_pre;     // [S + 1] key units of the row kernel's sequences before each (one kv head)
  int32_t* blk_seq;     // [blocks] sequence of each 256-row block of the tile kernel
  int32_t* blk_row;     // [blocks]   its first row (token * G + head of the group) in the sequence
  int64_t* blk_pre;     // [blocks + 1] key tiles of the blocks before each (one kv head)
  int32_t* counts;      // [0] blocks of the tile kernel, [1] first rejected sequence (INT32_MAX if none)
  uint32_t* sync;       // [row_ctas] arrivals of the row kernel's split items (zero between launches)
  uint32_t* tile_sync;  // [2 tile_ctas] of the tile kernel's, one for each 128-row tile
  uint32_t* err;        // device error word (ptx::kErr* bits)
  float* part;          // partial results of the row kernel's split items
  float* tile_part;     // of the tile kernel's
  int S, T, max_pages, Hq, Hkv, G, hd;
  int row_limit;        // rows (new tokens * G) up to which a sequence takes the row kernel
  int row_ctas, tile_ctas;
};

// Keys of one unit of the row kernel (four warps x 16 keys) and of one tile of the tile kernel;
// rows of one block of the tile kernel.
constexpr int kRowUnit = 64;
constexpr int kTileKeys = 128;
constexpr int kBlockRows = 256;

// Per-pair rotation frequencies in turns per position, each as a sum of two floats.
struct RopeView {
  const float2* freq;   // [rot / 2]
  int rot;              // rotated elements of a head (0: none)
  int interleaved;      // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  float mscale;         // factor on cos and sin
};

cudaError_t launch_build_seq(const int32_t* q_start, const int32_t* kv_len, const int32_t* pages, int table_ld,
                             const SeqView& s, int max_new, const KvView& kv, cudaStream_t st);
cudaError_t launch_qkv_write(const float* qkv, int64_t ld, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                             const RopeView& rope, const int32_t* positions, uint16_t* q, const KvView& kv,
                             const SeqView& s, int num_sms, cudaStream_t st);
cudaError_t launch_kv_read(const int32_t* row_start, int64_t rows, uint16_t* k, uint16_t* v, const KvView& kv,
                           const SeqView& s, int num_sms, cudaStream_t st);
// Sequences of at most SeqView::row_limit rows (single tokens and short chunks), and the zero rows of
// tokens in no sequence.
cudaError_t launch_attention_rows(const uint16_t* q, uint16_t* o, float scale, const KvView& kv, const SeqView& s,
                                  cudaStream_t st);
// The other sequences; tk and tv: the maps of a bf16 cache's K and V (make_kv_maps; not read for e4m3).
cudaError_t launch_attention_tiles(const CUtensorMap& tk, const CUtensorMap& tv, const uint16_t* q, uint16_t* o,
                                   float scale, const KvView& kv, const SeqView& s, cudaStream_t st);
// K and V as matrices [n_pages * Hkv * page, hd] in boxes of min(page, 128) rows x 64 columns.
bool make_kv_maps(const KvView& kv, CUtensorMap* k, CUtensorMap* v);
// Bytes of the partial results: two of 16 rows for each CTA of the row kernel, two of two 128-row tiles for each
// CTA of the tile kernel.
inline size_t row_part_bytes(const SeqView& s) { return static_cast<size_t>(s.row_ctas) * 2 * 16 * (s.hd + 2) * 4; }
inline size_t tile_part_bytes(const SeqView& s) { return static_cast<size_t>(s.tile_ctas) * 2 * 2 * 128 * (s.hd + 2) * 4; }

}  // namespace mlora
