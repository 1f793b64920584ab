// Host side of the attention step behind mlora.h: the paged KV cache, the rotation, a step's
// sequences, argument checks and dispatch.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <new>

#include "attention.h"
#include "internal.h"
#include "mlora.h"
#include "ptx.cuh"

using namespace mlora;

namespace {

template <typename... A>
mlora_status fail(mlora_status st, const char* fmt, A... a) {
  char buf[512];
  snprintf(buf, sizeof buf, fmt, a...);
  return report_error(st, buf);
}
mlora_status fail(mlora_status st, const char* text) { return report_error(st, text); }

#define ATTN_CUDA(call, what)                                  \
  do {                                                         \
    cudaError_t e__ = (call);                                  \
    if (e__ != cudaSuccess) return report_cuda_error(e__, what); \
  } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mlora_status created(cudaError_t e, const char* what) {
  cudaGetLastError();
  if (e == cudaErrorMemoryAllocation) return fail(MLORA_ERR_OOM, "%s: out of device memory", what);
  return report_cuda_error(e, what);
}

mlora_status check_cache_sizes(int n_pages, int page, int n_kv_heads, int hd, int type) {
  if (type != MLORA_KV_BF16 && type != MLORA_KV_E4M3)
    return fail(MLORA_ERR_INVALID_ARG, "cache type %d is neither MLORA_KV_BF16 nor MLORA_KV_E4M3", type);
  if (page < 8 || page > 256 || (page & (page - 1)))
    return fail(MLORA_ERR_INVALID_ARG, "page size %d must be 8, 16, 32, 64, 128 or 256", page);
  if (hd != 64 && hd != 128) return fail(MLORA_ERR_INVALID_ARG, "head size %d must be 64 or 128", hd);
  if (n_kv_heads < 1 || n_kv_heads > MLORA_MAX_HEADS)
    return fail(MLORA_ERR_INVALID_ARG, "%d key/value heads outside [1, %d]", n_kv_heads, MLORA_MAX_HEADS);
  if (n_pages < 1 || static_cast<int64_t>(n_pages) * page * n_kv_heads > INT32_MAX)
    return fail(MLORA_ERR_INVALID_ARG, "n_pages %d must be positive, and n_pages * page size * heads below 2^31", n_pages);
  return MLORA_OK;
}

}  // namespace

struct mlora_kv {
  KvView view{};
  bool own = false;
  CUtensorMap map_k{}, map_v{};
};

struct mlora_rope {
  float4* freq = nullptr;
  int rot = 0, interleaved = 0;
  float mscale = 1.f;
};

struct mlora_seq {
  SeqView view{};
  SeqView prefix{};                   // of the pass over shared prefixes: its lists beside the step's
  int max_groups = 0;
  bool prefixes = false;              // the last build has such a pass
  int32_t *skip = nullptr, *group = nullptr;
  int2* pre_at = nullptr;
  int max_seqs = 0, max_tokens = 0, num_sms = 0;
  int64_t max_blocks = 0;
  void* mem = nullptr;
  bool built = false;
  int page = 0, n_pages = 0, type = 0;   // of the cache that the last build checked its tables against
  bool tiles = false;                 // the last build may hold sequences above the row limit
  cudaEvent_t done = nullptr;
  cudaStream_t last_stream = nullptr;
};

extern "C" {

// ---------------------------------------------------------------- the paged cache
size_t mlora_kv_bytes(int n_pages, int page_size, int n_kv_heads, int head_dim, int type) {
  if (check_cache_sizes(n_pages, page_size, n_kv_heads, head_dim, type)) return 0;
  const size_t rows = static_cast<size_t>(n_pages) * page_size * n_kv_heads;
  return 2 * rows * (type == MLORA_KV_BF16 ? static_cast<size_t>(head_dim) * 2 : static_cast<size_t>(head_dim) + 4);
}

mlora_status mlora_kv_create(int n_pages, int page_size, int n_kv_heads, int head_dim, int type, void* K, void* V,
                             float* k_scale, float* v_scale, mlora_kv_t* out) {
  if (!out) return fail(MLORA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (mlora_status st = check_cache_sizes(n_pages, page_size, n_kv_heads, head_dim, type)) return st;
  const bool scales = type == MLORA_KV_E4M3;
  const bool own = !K && !V && !k_scale && !v_scale;
  if (!own) {
    if (!K || !V || (scales && (!k_scale || !v_scale)) || (!scales && (k_scale || v_scale)))
      return fail(MLORA_ERR_INVALID_ARG, "give K and V, and both scales for an e4m3 cache alone, or none of them");
    if (!aligned(K, 16) || !aligned(V, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16))
      return fail(MLORA_ERR_INVALID_ARG, "the cache's arrays must be 16-byte aligned");
  }
  mlora_kv* kv = new (std::nothrow) mlora_kv();
  if (!kv) return fail(MLORA_ERR_OOM, "host allocation failed");
  KvView& w = kv->view;
  w.n_pages = n_pages;
  w.page = page_size;
  w.page_log2 = 0;
  while ((1 << w.page_log2) < page_size) ++w.page_log2;
  w.Hkv = n_kv_heads;
  w.hd = head_dim;
  w.type = type;
  w.K = K, w.V = V, w.k_scale = k_scale, w.v_scale = v_scale;
  kv->own = own;
  if (own) {
    const size_t rows = static_cast<size_t>(n_pages) * page_size * n_kv_heads;
    const size_t bytes = rows * head_dim * (scales ? 1 : 2);
    cudaError_t e = cudaMalloc(&w.K, bytes);
    if (e == cudaSuccess) e = cudaMalloc(&w.V, bytes);
    if (e == cudaSuccess && scales) e = cudaMalloc(reinterpret_cast<void**>(&w.k_scale), rows * 4);
    if (e == cudaSuccess && scales) e = cudaMalloc(reinterpret_cast<void**>(&w.v_scale), rows * 4);
    if (e == cudaSuccess) e = cudaMemset(w.K, 0, bytes);
    if (e == cudaSuccess) e = cudaMemset(w.V, 0, bytes);
    if (e == cudaSuccess && scales) e = cudaMemset(w.k_scale, 0, rows * 4);
    if (e == cudaSuccess && scales) e = cudaMemset(w.v_scale, 0, rows * 4);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
      mlora_kv_destroy(kv);
      return created(e, "KV cache");
    }
  }
  if (!make_kv_maps(w, &kv->map_k, &kv->map_v)) {
    mlora_kv_destroy(kv);
    return fail(MLORA_ERR_CUDA, "tensor maps of the cache");
  }
  *out = kv;
  return MLORA_OK;
}

mlora_status mlora_kv_destroy(mlora_kv_t kv) {
  if (!kv) return MLORA_OK;
  if (kv->own) {
    cudaFree(kv->view.K);
    cudaFree(kv->view.V);
    cudaFree(kv->view.k_scale);
    cudaFree(kv->view.v_scale);
  }
  delete kv;
  return MLORA_OK;
}

mlora_status mlora_kv_info(mlora_kv_t kv, int* n_pages, int* page_size, int* n_kv_heads, int* head_dim, int* type,
                           void** K, void** V, void** k_scale, void** v_scale) {
  if (!kv) return fail(MLORA_ERR_INVALID_ARG, "cache is NULL");
  const KvView& w = kv->view;
  if (n_pages) *n_pages = w.n_pages;
  if (page_size) *page_size = w.page;
  if (n_kv_heads) *n_kv_heads = w.Hkv;
  if (head_dim) *head_dim = w.hd;
  if (type) *type = w.type;
  if (K) *K = w.K;
  if (V) *V = w.V;
  if (k_scale) *k_scale = w.k_scale;
  if (v_scale) *v_scale = w.v_scale;
  return MLORA_OK;
}

// ---------------------------------------------------------------- rotary positions
mlora_status mlora_rope_frequencies(int rot_dim, double theta, int scaling, double factor, double original_len,
                                    double low, double high, double* freq) {
  if (!freq) return fail(MLORA_ERR_INVALID_ARG, "freq is NULL");
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 256) return fail(MLORA_ERR_INVALID_ARG, "rot_dim %d must be even, in [2, 256]", rot_dim);
  if (!(theta > 1.0) || !std::isfinite(theta)) return fail(MLORA_ERR_INVALID_ARG, "theta must be above 1 and finite");
  if (scaling < MLORA_ROPE_PLAIN || scaling > MLORA_ROPE_RAMP) return fail(MLORA_ERR_INVALID_ARG, "unknown scaling %d", scaling);
  if (scaling != MLORA_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
    return fail(MLORA_ERR_INVALID_ARG, "factor must be at least 1 and finite");
  if (scaling == MLORA_ROPE_BASE && rot_dim < 4) return fail(MLORA_ERR_INVALID_ARG, "base scaling needs rot_dim >= 4");
  if (scaling >= MLORA_ROPE_WAVES && !(original_len > 0.0 && std::isfinite(original_len) && low > 0.0 && high > low && std::isfinite(high)))
    return fail(MLORA_ERR_INVALID_ARG, "original_len must be positive and 0 < low < high");
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  const int half = rot_dim / 2;
  const double base = scaling == MLORA_ROPE_BASE ? theta * std::pow(factor, rot_dim / (rot_dim - 2.0)) : theta;
  // RAMP: pair indices at which a frequency turns `high` (fast) and `low` times over the original length
  auto pair_of = [&](double turns) { return rot_dim * std::log(original_len / (turns * kTwoPi)) / (2.0 * std::log(theta)); };
  double fast = 0.0, slow = 0.0;
  if (scaling == MLORA_ROPE_RAMP) {
    fast = std::fmax(std::floor(pair_of(high)), 0.0);
    slow = std::fmin(std::ceil(pair_of(low)), rot_dim - 1.0);
    if (slow <= fast) slow = fast + 1e-3;
  }
  for (int i = 0; i < half; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double keep = 1.0;                       // share of the unscaled frequency
    if (scaling == MLORA_ROPE_LINEAR) keep = 0.0;
    if (scaling == MLORA_ROPE_WAVES) {
      const double turns = original_len * f / kTwoPi;
      keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
    }
    if (scaling == MLORA_ROPE_RAMP) keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - fast) / (slow - fast)));
    freq[i] = scaling == MLORA_ROPE_PLAIN || scaling == MLORA_ROPE_BASE ? f : f * (keep + (1.0 - keep) / factor);
  }
  return MLORA_OK;
}

mlora_status mlora_rope_create(int rot_dim, int interleaved, const double* freq, float mscale, mlora_rope_t* out) {
  if (!out) return fail(MLORA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (rot_dim < 8 || rot_dim % 8 || rot_dim > 128) return fail(MLORA_ERR_INVALID_ARG, "rot_dim %d must be a multiple of 8 in [8, 128]", rot_dim);
  if (!freq) return fail(MLORA_ERR_INVALID_ARG, "freq is NULL");
  if (!std::isfinite(mscale)) return fail(MLORA_ERR_INVALID_ARG, "mscale must be finite");
  // Turns per position, freq / (2 pi), to twice a double's bits, as a sum of three floats: positions up to 2^24 times frequencies
  // up to 1e6 are 2^42 turns, of which the kernel wants 2^-24.
  constexpr double kTwoPi = 6.283185307179586476925286766559, kTwoPiRest = 2.4492935982947064e-16;      // their sum
  float4 host[64];
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!(std::fabs(freq[i]) <= 1e6)) return fail(MLORA_ERR_INVALID_ARG, "frequency %d is not a number of magnitude up to 1e6", i);
    const double turns = freq[i] / kTwoPi, rest = (std::fma(-turns, kTwoPi, freq[i]) - turns * kTwoPiRest) / kTwoPi;
    host[i].x = static_cast<float>(turns);
    const double y = (turns - static_cast<double>(host[i].x)) + rest;
    host[i].y = static_cast<float>(y);
    host[i].z = static_cast<float>(y - static_cast<double>(host[i].y));
    host[i].w = 0.f;
  }
  mlora_rope* r = new (std::nothrow) mlora_rope();
  if (!r) return fail(MLORA_ERR_OOM, "host allocation failed");
  r->rot = rot_dim;
  r->interleaved = interleaved != 0;
  r->mscale = mscale;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&r->freq), sizeof(float4) * rot_dim / 2);
  if (e == cudaSuccess) e = cudaMemcpy(r->freq, host, sizeof(float4) * rot_dim / 2, cudaMemcpyHostToDevice);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    mlora_rope_destroy(r);
    return created(e, "rotation");
  }
  *out = r;
  return MLORA_OK;
}

mlora_status mlora_rope_destroy(mlora_rope_t r) {
  if (!r) return MLORA_OK;
  cudaFree(r->freq);
  delete r;
  return MLORA_OK;
}

// ---------------------------------------------------------------- a step's sequences
mlora_status mlora_seq_create(int max_seqs, int max_tokens, int max_pages, int n_q_heads, int n_kv_heads, int head_dim,
                              mlora_seq_t* out) {
  return mlora_seq_create_groups(max_seqs, max_tokens, max_pages, n_q_heads, n_kv_heads, head_dim, 0, out);
}

mlora_status mlora_seq_create_groups(int max_seqs, int max_tokens, int max_pages, int n_q_heads, int n_kv_heads, int head_dim,
                                     int max_groups, mlora_seq_t* out) {
  if (!out) return fail(MLORA_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (max_seqs < 1 || max_seqs > MLORA_MAX_SEQS)
    return fail(MLORA_ERR_INVALID_ARG, "max_seqs %d outside [1, %d]", max_seqs, MLORA_MAX_SEQS);
  if (max_tokens < 1 || max_tokens > MLORA_MAX_TOKENS)
    return fail(MLORA_ERR_INVALID_ARG, "max_tokens %d outside [1, %d]", max_tokens, MLORA_MAX_TOKENS);
  if (max_pages < 1 || static_cast<int64_t>(max_pages) * max_seqs > (1 << 30))
    return fail(MLORA_ERR_INVALID_ARG, "max_pages %d must be positive, and max_pages * max_seqs at most 2^30", max_pages);
  if (head_dim != 64 && head_dim != 128) return fail(MLORA_ERR_INVALID_ARG, "head size %d must be 64 or 128", head_dim);
  if (n_kv_heads < 1 || n_kv_heads > MLORA_MAX_HEADS || n_q_heads < n_kv_heads || n_q_heads > MLORA_MAX_HEADS || n_q_heads % n_kv_heads)
    return fail(MLORA_ERR_INVALID_ARG, "%d query heads must be a multiple of %d key/value heads, both in [1, %d]", n_q_heads, n_kv_heads, MLORA_MAX_HEADS);
  if (n_q_heads / n_kv_heads > 128)
    return fail(MLORA_ERR_INVALID_ARG, "%d query heads for each key/value head, at most 128", n_q_heads / n_kv_heads);
  if (max_groups < 0 || max_groups > max_seqs)
    return fail(MLORA_ERR_INVALID_ARG, "max_groups %d outside [0, max_seqs = %d]", max_groups, max_seqs);
  int sms = 0;
  if (mlora_status st = device_sms(&sms)) return st;
  mlora_seq* q = new (std::nothrow) mlora_seq();
  if (!q) return fail(MLORA_ERR_OOM, "host allocation failed");
  q->max_seqs = max_seqs;
  q->max_tokens = max_tokens;
  q->num_sms = sms;
  SeqView& v = q->view;
  v.max_pages = max_pages;
  v.Hq = n_q_heads;
  v.Hkv = n_kv_heads;
  v.G = n_q_heads / n_kv_heads;
  v.tile_tokens = 128 / v.G;
  v.hd = head_dim;
  v.row_ctas = 3 * sms;               // at most (mlora_build_seq)
  v.tile_ctas = sms;
  q->max_groups = max_groups;
  const size_t S = max_seqs, T = max_tokens, N = max_groups;
  q->max_blocks = most_blocks(v, T, S);
  const size_t J = q->max_blocks, P = N > 0 ? most_blocks(v, T, N) : 0;      // P: blocks of the prefix pass
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t R = v.row_ctas, C = v.tile_ctas;
  const size_t o_start = take(S * 4), o_n = take(S * 4), o_len = take(S * 4), o_table = take(S * max_pages * 4),
               o_seq = take(T * 4), o_pos = take(T * 4), o_row = take(T * 4), o_pp = take((S + 1) * 4),
               o_rs = take(S * sizeof(RowSeq)), o_rp = take((S + 1) * 8), o_blk = take(J * sizeof(TileBlk)),
               o_bp = take((J + 1) * 8), o_rsh = take(R * sizeof(RowShare)), o_tsh = take(C * sizeof(int2)), o_tw = take((J * n_kv_heads + C) * sizeof(TileWork)),
               o_there = take(3 * R * 4), o_tj = take(C * sizeof(JoinTask)), o_counts = take(8 * 4),
               o_err = take(4), o_gap = take(S * 4), o_part = take(row_part_bytes(v)), o_tile_part = take(tile_part_bytes(v));
  const size_t o_skip = take(N ? S * 4 : 0), o_group = take(N ? S * 4 : 0), o_at = take(N ? S * sizeof(int2) : 0), o_gs = take(N * 4),
               o_gn = take(N * 4), o_gl = take(N * 4), o_rep = take(N * 4), o_gb = take(N * 4), o_pblk = take(P * sizeof(TileBlk)),
               o_pbp = take((P + 1) * 8), o_ptsh = take(C * sizeof(int2)), o_ptw = take((P * n_kv_heads + C) * sizeof(TileWork)),
               o_ptj = take(C * sizeof(JoinTask)), o_pcounts = take(8 * 4),
               o_pre = take(P * n_kv_heads * 2 * static_cast<size_t>(tile_slot(v)) * 4);
  cudaError_t e = cudaMalloc(&q->mem, at);
  if (e == cudaSuccess) {
    char* b = static_cast<char*>(q->mem);
    v.start = reinterpret_cast<int32_t*>(b + o_start);
    v.n = reinterpret_cast<int32_t*>(b + o_n);
    v.len = reinterpret_cast<int32_t*>(b + o_len);
    v.table = reinterpret_cast<int32_t*>(b + o_table);
    v.tok_seq = reinterpret_cast<int32_t*>(b + o_seq);
    v.tok_pos = reinterpret_cast<int32_t*>(b + o_pos);
    v.tok_row = reinterpret_cast<int32_t*>(b + o_row);
    v.page_pre = reinterpret_cast<int32_t*>(b + o_pp);
    v.row_seq = reinterpret_cast<RowSeq*>(b + o_rs);
    v.row_pre = reinterpret_cast<int64_t*>(b + o_rp);
    v.blk = reinterpret_cast<TileBlk*>(b + o_blk);
    v.blk_pre = reinterpret_cast<int64_t*>(b + o_bp);
    v.row_share = reinterpret_cast<RowShare*>(b + o_rsh);
    v.tile_share = reinterpret_cast<int2*>(b + o_tsh);
    v.tile_work = reinterpret_cast<TileWork*>(b + o_tw);
    v.row_there = reinterpret_cast<int32_t*>(b + o_there);
    v.tile_join = reinterpret_cast<JoinTask*>(b + o_tj);
    v.counts = reinterpret_cast<int32_t*>(b + o_counts);
    v.err = reinterpret_cast<uint32_t*>(b + o_err);
    v.row_part = reinterpret_cast<float*>(b + o_part);
    v.tile_part = reinterpret_cast<float*>(b + o_tile_part);
    v.row_gap = reinterpret_cast<int32_t*>(b + o_gap);
    if (N > 0) {
      q->skip = reinterpret_cast<int32_t*>(b + o_skip);
      q->group = reinterpret_cast<int32_t*>(b + o_group);
      q->pre_at = reinterpret_cast<int2*>(b + o_at);
      v.pre_part = reinterpret_cast<float*>(b + o_pre);
      SeqView& p = q->prefix = v;
      p.start = reinterpret_cast<int32_t*>(b + o_gs);
      p.n = reinterpret_cast<int32_t*>(b + o_gn);
      p.len = reinterpret_cast<int32_t*>(b + o_gl);
      p.rep = reinterpret_cast<int32_t*>(b + o_rep);
      p.first_blk = reinterpret_cast<int32_t*>(b + o_gb);
      p.blk = reinterpret_cast<TileBlk*>(b + o_pblk);
      p.blk_pre = reinterpret_cast<int64_t*>(b + o_pbp);
      p.tile_share = reinterpret_cast<int2*>(b + o_ptsh);
      p.tile_work = reinterpret_cast<TileWork*>(b + o_ptw);
      p.tile_join = reinterpret_cast<JoinTask*>(b + o_ptj);
      p.counts = reinterpret_cast<int32_t*>(b + o_pcounts);
      p.see = kSeePrefix;
      p.window = INT_MAX;
      p.sinks = p.gap_chunk = p.gap_tile = 0;
    }
    const int32_t counts[8] = {0, INT32_MAX, 0, 0, 0, 0, 0, 0};
    e = cudaMemset(v.err, 0, 4);
    if (e == cudaSuccess) e = cudaMemcpy(v.counts, counts, sizeof counts, cudaMemcpyHostToDevice);
  }
  if (e == cudaSuccess) e = cudaEventCreateWithFlags(&q->done, cudaEventDisableTiming);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    mlora_seq_destroy(q);
    return created(e, "sequence metadata");
  }
  *out = q;
  return MLORA_OK;
}

mlora_status mlora_seq_destroy(mlora_seq_t q) {
  if (!q) return MLORA_OK;
  if (q->done) {
    if (q->built && cudaEventRecord(q->done, q->last_stream) == cudaSuccess) cudaEventSynchronize(q->done);
    cudaEventDestroy(q->done);
  }
  cudaFree(q->mem);
  delete q;
  return MLORA_OK;
}

static mlora_status build_seq(mlora_seq_t q, const int32_t* q_start, const int32_t* kv_len, const int32_t* pages, int pages_ld,
                              int n_seqs, int T, int max_new, int window, int sinks, const int32_t* group_start,
                              const int32_t* prefix_len, int n_groups, mlora_kv_t kv, void* stream) {
  if (n_seqs < 0 || T < 0 || max_new < 0) return fail(MLORA_ERR_INVALID_ARG, "n_seqs %d, T %d and max_new %d must be >= 0", n_seqs, T, max_new);
  if (n_seqs > q->max_seqs || T > q->max_tokens)
    return fail(MLORA_ERR_TOO_MANY_TOKENS, "%d sequences, %d tokens exceed the object's %d and %d", n_seqs, T, q->max_seqs, q->max_tokens);
  if (n_seqs > 0 && (!q_start || !kv_len || !pages)) return fail(MLORA_ERR_INVALID_ARG, "q_start, kv_len or pages is NULL");
  if (pages_ld < 1 || pages_ld < q->view.max_pages)
    return fail(MLORA_ERR_INVALID_ARG, "page table rows of %d entries, the object reads %d", pages_ld, q->view.max_pages);
  const KvView& w = kv->view;
  if (w.Hkv != q->view.Hkv || w.hd != q->view.hd)
    return fail(MLORA_ERR_MISMATCH, "the cache has %d heads of %d, the sequences' object %d of %d", w.Hkv, w.hd, q->view.Hkv, q->view.hd);
  SeqView& v = q->view;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  v.S = n_seqs;
  v.T = T;
  // Rows up to which a sequence takes the row kernel: 8, or 16 where no sequence has more than 16 rows
  // or a single token has more than 8.
  const int64_t most = static_cast<int64_t>(max_new) * v.G;
  v.row_limit = most <= 8 ? 8 : most <= 16 || v.G > 8 ? 16 : 8;
  v.row_ctas = rows_ctas_per_sm(v.row_limit > 8, w.type == kKvE4m3) * q->num_sms;
  v.see = window > 0 || n_groups > 0 ? kSeeRanges : kSeeAll;
  v.window = window > 0 ? window : INT_MAX;
  v.sinks = sinks;
  v.gap_chunk = (sinks + kRowChunk - 1) / kRowChunk;
  v.gap_tile = (sinks + kTileKeys - 1) / kTileKeys;
  v.skip = n_groups > 0 ? q->skip : nullptr;
  v.group = n_groups > 0 ? q->group : nullptr;
  v.pre_at = n_groups > 0 ? q->pre_at : nullptr;
  SeqReuse reuse{window, sinks, group_start, prefix_len, n_groups, q->prefix};
  reuse.prefix.S = n_groups;
  reuse.prefix.T = T;
  reuse.prefix.row_limit = v.row_limit;
  q->prefix = reuse.prefix;
  q->prefixes = n_groups > 0;
  q->tiles = most > v.row_limit;
  q->page = w.page;
  q->n_pages = w.n_pages;
  q->type = w.type;
  const cudaError_t e = launch_build_seq(q_start, kv_len, pages, pages_ld, v, max_new, w, reuse, s);
  if (e != cudaSuccess) return report_cuda_error(e, "build_seq launch");
  q->last_stream = s;
  q->built = true;
  return MLORA_OK;
}

mlora_status mlora_build_seq(mlora_seq_t q, const int32_t* q_start, const int32_t* kv_len, const int32_t* pages,
                             int pages_ld, int n_seqs, int T, int max_new, mlora_kv_t kv, void* stream) {
  if (!q || !kv) return fail(MLORA_ERR_INVALID_ARG, "seq or cache is NULL");
  return build_seq(q, q_start, kv_len, pages, pages_ld, n_seqs, T, max_new, 0, 0, nullptr, nullptr, 0, kv, stream);
}

mlora_status mlora_build_seq_window(mlora_seq_t q, const int32_t* q_start, const int32_t* kv_len, const int32_t* pages,
                                    int pages_ld, int n_seqs, int T, int max_new, int window, int sinks, mlora_kv_t kv,
                                    void* stream) {
  if (!q || !kv) return fail(MLORA_ERR_INVALID_ARG, "seq or cache is NULL");
  if (window < 1) return fail(MLORA_ERR_INVALID_ARG, "window %d must be positive", window);
  if (sinks < 0 || sinks > MLORA_MAX_SINKS) return fail(MLORA_ERR_INVALID_ARG, "sinks %d outside [0, %d]", sinks, MLORA_MAX_SINKS);
  return build_seq(q, q_start, kv_len, pages, pages_ld, n_seqs, T, max_new, window, sinks, nullptr, nullptr, 0, kv, stream);
}

// Whether a pass over prefixes of up to max_prefix keys may save more than it costs: two launches, and the rows' fp32 sums written
// and read again. What it saves: where single tokens and other few rows take the row kernel, the reads of all sequences of a group
// but one, mostly from L2; where the rows take the tile kernel, blocks of key tiles, as far as the sequences' own blocks are not
// full. (Graph times without and with a pass. One token each behind 4100, 8 heads of 128: 8 of them, bf16, 17.6 and 20.6 us; 16, 26.3
// and 20.5; e4m3 16, 25.7 and 27.9; 64, 77.6 and 34.5. 16 chunks behind 9000, 32 heads on 8: of 8 tokens 108 and 38 us, of 48 126 and
// 112, of 64, a full block each, 135 and 139, of 96 222 and 194, of 128 229 and 240; e4m3 170 and 53, 196 and 172, 210 and 219, ...)
static bool sharing_pays(const SeqView& v, const KvView& w, int num_sms, int n_seqs, int T, int max_new, int n_groups, int max_prefix) {
  constexpr double kL2 = 13e6, kSums = 5e6;                       // bytes a us
  double cost = 10.0;                                             // us; with few items, whose keys are split finely, more:
  const bool e4m3 = w.type == kKvE4m3;
  const double keys = static_cast<double>(std::min(static_cast<int64_t>(max_prefix), static_cast<int64_t>(v.max_pages) * w.page));
  double saved = 0.0;
  if (static_cast<int64_t>(max_new) * v.G <= 16) {
    saved = std::max(n_seqs - n_groups, 0) * keys * w.Hkv * 2 * w.hd * (e4m3 ? 1 : 2) / kL2;
  } else if (n_seqs > 0) {
    const double per = 2 * v.tile_tokens, mean = static_cast<double>(T) / n_seqs;
    const double apart = n_seqs * std::ceil(mean / per), together = T / per + n_groups;
    cost = 20.0;                                                  // (e4m3, 16 heads on 1, 2 tokens behind 9000: 33 us, 48 with a pass)
    saved = std::max(apart - together, 0.0) * w.Hkv * keys / kTileKeys * (e4m3 ? 2.8 : 1.45) / num_sms;      // us of a key tile on an SM
  }
  return T > 0 && saved > cost + static_cast<double>(T) * v.Hq * (w.hd + 2) * 8 / kSums;
}

mlora_status mlora_build_seq_groups(mlora_seq_t q, const int32_t* q_start, const int32_t* kv_len, const int32_t* pages,
                                    int pages_ld, int n_seqs, int T, int max_new, const int32_t* group_start,
                                    const int32_t* prefix_len, int n_groups, int max_prefix, mlora_kv_t kv, void* stream) {
  if (!q || !kv) return fail(MLORA_ERR_INVALID_ARG, "seq or cache is NULL");
  if (n_groups < 0 || max_prefix < 0) return fail(MLORA_ERR_INVALID_ARG, "n_groups %d and max_prefix %d must be >= 0", n_groups, max_prefix);
  if (n_groups > q->max_groups)
    return fail(MLORA_ERR_TOO_MANY_TOKENS, "%d groups exceed the object's %d", n_groups, q->max_groups);
  if (n_groups > 0 && (!group_start || !prefix_len)) return fail(MLORA_ERR_INVALID_ARG, "group_start or prefix_len is NULL");
  if (n_groups > 0 && !sharing_pays(q->view, kv->view, q->num_sms, n_seqs, T, max_new, n_groups, max_prefix)) n_groups = 0;
  return build_seq(q, q_start, kv_len, pages, pages_ld, n_seqs, T, max_new, 0, 0, group_start, prefix_len, n_groups, kv, stream);
}

mlora_status mlora_seq_status(mlora_seq_t q) {
  if (!q) return fail(MLORA_ERR_INVALID_ARG, "seq is NULL");
  if (!q->built) return MLORA_OK;
  ATTN_CUDA(cudaEventRecord(q->done, q->last_stream), "record sequence event");
  ATTN_CUDA(cudaEventSynchronize(q->done), "sequence sync");
  uint32_t err = 0;
  int32_t first = 0;
  ATTN_CUDA(cudaMemcpy(&err, q->view.err, 4, cudaMemcpyDeviceToHost), "read sequence error word");
  if (!err) return MLORA_OK;
  const int32_t none = INT32_MAX;
  ATTN_CUDA(cudaMemcpy(&first, q->view.counts + 1, 4, cudaMemcpyDeviceToHost), "read sequence counts");
  ATTN_CUDA(cudaMemcpy(q->view.counts + 1, &none, 4, cudaMemcpyHostToDevice), "clear sequence counts");
  ATTN_CUDA(cudaMemset(q->view.err, 0, 4), "clear sequence error word");
  if (err & ptx::kErrWaitTimeout) return fail(MLORA_ERR_DEVICE_TIMEOUT, "a kernel's bounded wait timed out");
  if (err & ptx::kErrBadSeq)
    return fail(MLORA_ERR_BAD_SEQUENCE, "sequence %d: its tokens, length or pages do not hold; it was skipped", first);
  if (err & ptx::kErrBadGroups)
    return fail(MLORA_ERR_INVALID_ARG, "the groups' bounds do not ascend within the sequences: none was shared");
  return fail(MLORA_ERR_INVALID_ARG, "a cache read's rows lie outside its output");
}

static mlora_status check_step(mlora_kv_t kv, mlora_seq_t q) {
  if (!kv || !q) return fail(MLORA_ERR_INVALID_ARG, "cache or seq is NULL");
  if (!q->built) return fail(MLORA_ERR_INVALID_ARG, "the sequences have not been built");
  const KvView& w = kv->view;
  if (w.Hkv != q->view.Hkv || w.hd != q->view.hd)
    return fail(MLORA_ERR_MISMATCH, "the cache has %d heads of %d, the sequences' object %d of %d", w.Hkv, w.hd, q->view.Hkv, q->view.hd);
  if (w.page != q->page || w.n_pages != q->n_pages)
    return fail(MLORA_ERR_MISMATCH, "the sequences were built on a cache of %d pages of %d, this one has %d of %d", q->n_pages, q->page, w.n_pages, w.page);
  if (w.type != q->type) return fail(MLORA_ERR_MISMATCH, "the sequences were built on a cache of another element type");
  return MLORA_OK;
}

// ---------------------------------------------------------------- the operators
mlora_status mlora_qkv_write(mlora_kv_t kv, mlora_seq_t q, const float* qkv, int64_t ld, const mlora_bf16* q_norm,
                             const mlora_bf16* k_norm, float eps, mlora_rope_t rope, const int32_t* positions,
                             mlora_bf16* q_out, void* stream) {
  if (mlora_status st = check_step(kv, q)) return st;
  const SeqView& v = q->view;
  const int64_t width = static_cast<int64_t>(v.Hq + 2 * v.Hkv) * v.hd;
  if (ld < width || ld % 4) return fail(MLORA_ERR_INVALID_ARG, "qkv rows of %lld elements must be a multiple of 4 and at least %lld", (long long)ld, (long long)width);
  if (v.T > 0 && (!qkv || !q_out)) return fail(MLORA_ERR_INVALID_ARG, "qkv or q_out is NULL");
  if (!aligned(qkv, 16) || !aligned(q_out, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16))
    return fail(MLORA_ERR_INVALID_ARG, "qkv, q_out and the norms' weights must be 16-byte aligned");
  if ((q_norm || k_norm) && !(eps >= 0.f && std::isfinite(eps))) return fail(MLORA_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (rope && rope->rot > v.hd) return fail(MLORA_ERR_MISMATCH, "the rotation turns %d elements of heads of %d", rope->rot, v.hd);
  RopeView r{nullptr, 0, 0, 1.f};
  if (rope) r = RopeView{rope->freq, rope->rot, rope->interleaved, rope->mscale};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_qkv_write(qkv, ld, q_norm, k_norm, eps, r, positions, q_out, kv->view, v, q->num_sms, s);
  if (e != cudaSuccess) return report_cuda_error(e, "qkv write launch");
  q->last_stream = s;
  return MLORA_OK;
}

mlora_status mlora_attention(mlora_kv_t kv, mlora_seq_t q, const mlora_bf16* query, float scale, mlora_bf16* out,
                             void* stream) {
  if (mlora_status st = check_step(kv, q)) return st;
  const SeqView& v = q->view;
  if (v.T > 0 && (!query || !out)) return fail(MLORA_ERR_INVALID_ARG, "query or out is NULL");
  if (!aligned(query, 16) || !aligned(out, 16)) return fail(MLORA_ERR_INVALID_ARG, "query and out must be 16-byte aligned");
  if (!(scale > 0.f && std::isfinite(scale))) return fail(MLORA_ERR_INVALID_ARG, "scale must be positive and finite");
  const uintptr_t qa = reinterpret_cast<uintptr_t>(query), oa = reinterpret_cast<uintptr_t>(out);
  const uintptr_t bytes = static_cast<uintptr_t>(v.T) * v.Hq * v.hd * 2;
  if (qa < oa + bytes && oa < qa + bytes) return fail(MLORA_ERR_INVALID_ARG, "query and out must not overlap");
  if (v.T == 0) return MLORA_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (q->prefixes) {
    e = launch_attention_tiles(kv->map_k, kv->map_v, query, out, scale, kv->view, q->prefix, s);
    if (e == cudaSuccess) e = launch_attention_join(out, q->prefix, s);
  }
  if (e == cudaSuccess) e = launch_attention_rows(query, out, scale, kv->view, v, s);
  if (e == cudaSuccess && q->tiles) e = launch_attention_tiles(kv->map_k, kv->map_v, query, out, scale, kv->view, v, s);
  if (e == cudaSuccess && q->tiles) e = launch_attention_join(out, v, s);
  if (e != cudaSuccess) return report_cuda_error(e, "attention launch");
  q->last_stream = s;
  return MLORA_OK;
}

mlora_status mlora_kv_read(mlora_kv_t kv, mlora_seq_t q, const int32_t* row_start, int64_t rows, mlora_bf16* k_out,
                           mlora_bf16* v_out, void* stream) {
  if (mlora_status st = check_step(kv, q)) return st;
  if (rows < 0) return fail(MLORA_ERR_INVALID_ARG, "rows must be >= 0");
  if (q->view.S > 0 && !row_start) return fail(MLORA_ERR_INVALID_ARG, "row_start is NULL");
  if (rows > 0 && (!k_out || !v_out)) return fail(MLORA_ERR_INVALID_ARG, "k_out or v_out is NULL");
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return fail(MLORA_ERR_INVALID_ARG, "k_out and v_out must be 16-byte aligned");
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_kv_read(row_start, rows, k_out, v_out, kv->view, q->view, q->num_sms, s);
  if (e != cudaSuccess) return report_cuda_error(e, "cache read launch");
  q->last_stream = s;
  return MLORA_OK;
}

}  // extern "C"
