"""Torch-facing convenience objects over the C ABI (argument marshalling only).

``AdapterPool`` owns one adapted linear's slot pool, ``StepMeta`` one step's slot
metadata, and ``linear`` runs the layer y = x W^T + sum_j s c B(A x) into an fp32 tensor.
Torch provides device memory and streams; every step of the computation runs in
libmlora.so.
"""
from __future__ import annotations

import numpy as np
import torch

from . import mlora


def bf16_from_bits(bits: np.ndarray, device=None) -> torch.Tensor:
    """A bf16 tensor holding the given 16-bit patterns (numpy uint16)."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t.to(device) if device is not None else t


def _pinned_bits(a) -> torch.Tensor:
    if isinstance(a, torch.Tensor):
        t = a.detach().contiguous().cpu().view(torch.int16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16))
    return t.pin_memory() if torch.cuda.is_available() else t


class AdapterPool:
    """The slots of one adapted linear: A [C, K] and B [D, C] (bf16, zero padded) over a column
    space in which slot s owns its rank rows. With `classes` = [(n_slots_c, rank_c), ...] the slots
    come in rank classes (numbered class by class); otherwise n_slots slots of rank r_max."""

    def __init__(self, n_slots: int, r_max: int, K: int, D: int, copy_stream=None, classes=None):
        self.K, self.D = K, D
        if classes:
            self.classes = [(int(n), int(r)) for n, r in classes]
            self.n_slots = sum(n for n, _ in self.classes)
            self.r_max = max(r for _, r in self.classes)
            self.handle = mlora.mlora_pool_create_classes([n for n, _ in self.classes], [r for _, r in self.classes],
                                                          K, D, copy_stream)
        else:
            self.classes = None
            self.n_slots, self.r_max = n_slots, r_max
            self.handle = mlora.mlora_pool_create(n_slots, r_max, K, D, copy_stream)
        self._staged = []           # pinned host copies kept alive until the next sync

    def load(self, slot: int, A, B, rank: int, alpha: float, rslora: bool = False) -> None:
        a, b = _pinned_bits(A), _pinned_bits(B)
        assert a.numel() == rank * self.K and b.numel() == self.D * rank
        self._staged += [a, b]
        mlora.mlora_load_adapter(self.handle, slot, a.data_ptr(), b.data_ptr(), rank, alpha, rslora)

    def clear(self, slot: int) -> None:
        mlora.mlora_clear_slot(self.handle, slot)

    def sync(self) -> None:
        mlora.mlora_pool_sync(self.handle)
        self._staged.clear()

    def info(self) -> dict:
        return mlora.mlora_pool_info(self.handle)

    def layout(self) -> dict:
        return mlora.mlora_pool_layout(self.handle, self.n_slots)

    def close(self) -> None:
        if self.handle:
            mlora.mlora_pool_destroy(self.handle)
            self.handle = 0
            self._staged.clear()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class EmbeddingPool(AdapterPool):
    """The slots of an embedding table with LoRA: A kept token-major ([vocab, C]), B [dim, C].
    load() takes each adapter's A [rank, vocab] and B [dim, rank], like a linear pool with
    K = vocab and D = dim."""

    def __init__(self, vocab: int, dim: int, classes, copy_stream=None):
        self.K, self.D = vocab, dim
        self.classes = [(int(n), int(r)) for n, r in classes]
        self.n_slots = sum(n for n, _ in self.classes)
        self.r_max = max(r for _, r in self.classes)
        self.handle = mlora.mlora_embedding_pool_create([n for n, _ in self.classes], [r for _, r in self.classes],
                                                        vocab, dim, copy_stream)
        self._staged = []


class StepMeta:
    """Per-step slot metadata for up to max_tokens tokens with J slots each."""

    def __init__(self, max_tokens: int, J: int, r_max: int):
        self.max_tokens, self.J_max, self.r_max = max_tokens, J, r_max
        self.handle = mlora.mlora_meta_create(max_tokens, J, r_max)
        self.T = 0
        self.J = J

    def build(self, token_slots: torch.Tensor, scales: torch.Tensor | None, pool: AdapterPool, stream=None) -> None:
        assert token_slots.is_cuda and token_slots.dtype == torch.int32 and token_slots.is_contiguous()
        T, J = (token_slots.shape[0], token_slots.shape[1]) if token_slots.dim() == 2 else (token_slots.shape[0], 1)
        if scales is not None:
            assert scales.is_cuda and scales.dtype == torch.float32 and scales.numel() == T * J
        mlora.mlora_build_meta(self.handle, token_slots, scales, T, J, pool.handle, _stream(stream))
        self.T, self.J = T, J

    def status(self) -> None:
        mlora.mlora_meta_status(self.handle)

    def read(self) -> dict:
        return mlora.mlora_meta_read(self.handle, self.T * self.J)

    def close(self) -> None:
        if self.handle:
            mlora.mlora_meta_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream()
    return stream


def _torch_stream(stream, device: torch.device):
    """The torch stream of a torch stream or raw handle."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)


def _output(shape, dtype, device: torch.device, stream) -> torch.Tensor:
    """A new tensor for a call on `stream`. It is made there, so that nothing queued earlier on the current stream still works in
    its memory, and, once released, kept from reuse until what the current stream then has queued is done with it too."""
    here = None if stream is None else torch.cuda.current_stream(device)
    if here is None or here.cuda_stream == getattr(stream, "cuda_stream", stream):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_torch_stream(stream, device)):
        y = torch.empty(shape, dtype=dtype, device=device)
    y.record_stream(here)
    return y


# The current stream's raw handle. The attention step's calls take a few microseconds on the GPU for small batches, where
# making a Stream object for each (about 3 us) is felt.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device: torch.device):
    if stream is not None:
        return stream
    if _raw_current_stream is None:
        return torch.cuda.current_stream(device)
    return _raw_current_stream(device.index)


def linear(pool: AdapterPool, meta: StepMeta, x: torch.Tensor, W: torch.Tensor, y: torch.Tensor | None = None,
           stream=None) -> torch.Tensor:
    """y[T, D] fp32 = x W^T + the step's LoRA side path (x [T, K] and W [D, K] bf16 on the GPU)."""
    assert x.dtype == torch.bfloat16 and W.dtype == torch.bfloat16 and x.is_contiguous() and W.is_contiguous()
    T = meta.T
    assert x.shape == (T, pool.K) and W.shape == (pool.D, pool.K)
    if y is None:
        y = _output((T, pool.D), torch.float32, x.device, stream)
    mlora.mlora_linear(pool.handle, meta.handle, x, W, y, _stream(stream))
    return y


def embedding(pool: EmbeddingPool, meta: StepMeta, ids: torch.Tensor, E: torch.Tensor, y: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """y[T, dim] fp32 = E[ids] + the step's LoRA side path (ids int32 [T], E [vocab, dim] bf16 on the GPU)."""
    assert ids.dtype == torch.int32 and E.dtype == torch.bfloat16 and ids.is_contiguous() and E.is_contiguous()
    T = meta.T
    assert ids.shape == (T,) and E.shape == (pool.K, pool.D)
    if y is None:
        y = _output((T, pool.D), torch.float32, E.device, stream)
    mlora.mlora_embedding(pool.handle, meta.handle, ids, E, y, _stream(stream))
    return y


def base_gemm(x: torch.Tensor, W: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    T, K = x.shape
    D = W.shape[0]
    if y is None:
        y = _output((T, D), torch.float32, x.device, stream)
    mlora.mlora_base_gemm(x, W, y, T, K, D, _stream(stream))
    return y


# --------------------------------------------------------------------------------------- attention step
class KVCache:
    """The paged cache of one attention layer: k, v [n_pages, n_kv_heads, page_size, head_dim], bf16 or
    float8_e4m3fn with fp32 scales k_scale, v_scale [n_pages, n_kv_heads, page_size]. The tensors may be given
    (they then decide the type); otherwise they are made here, zeroed, of `dtype`."""

    def __init__(self, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, dtype=torch.bfloat16, k=None,
                 v=None, k_scale=None, v_scale=None, device="cuda"):
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        if k is None:
            assert v is None and k_scale is None and v_scale is None
            k, v = (torch.zeros(shape, dtype=torch.bfloat16, device=device) if dtype == torch.bfloat16 else
                    torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
            if dtype == torch.float8_e4m3fn:
                k_scale, v_scale = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
        assert k.dtype in (torch.bfloat16, torch.float8_e4m3fn) and v.dtype == k.dtype
        for x in (k, v):
            assert x.is_cuda and x.is_contiguous() and x.shape == shape
        e4m3 = k.dtype == torch.float8_e4m3fn
        assert (k_scale is not None) == e4m3 and (v_scale is not None) == e4m3
        for x in (k_scale, v_scale):
            assert x is None or (x.is_cuda and x.is_contiguous() and x.dtype == torch.float32 and x.shape == shape[:3])
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = n_pages, page_size, n_kv_heads, head_dim
        self.handle = mlora.mlora_kv_create(n_pages, page_size, n_kv_heads, head_dim,
                                            mlora.MLORA_KV_E4M3 if e4m3 else mlora.MLORA_KV_BF16, k, v, k_scale, v_scale)

    def close(self) -> None:
        if self.handle:
            mlora.mlora_kv_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Rope:
    """Rotary positions over the first rot_dim elements of each head: frequencies theta^(-2i / rot_dim), scaled by
    `scaling` = one of mlora.MLORA_ROPE_* with its keyword arguments (factor, original_len, low, high), or given whole
    as `freq` (radians per position)."""

    def __init__(self, rot_dim: int, theta: float = 10000.0, interleaved: bool = False, scaling: int = 0,
                 mscale: float = 1.0, freq=None, **kw):
        self.freq = mlora.mlora_rope_frequencies(rot_dim, theta, scaling, **kw) if freq is None else list(freq)
        self.rot_dim, self.interleaved, self.mscale = rot_dim, interleaved, mscale
        self.handle = mlora.mlora_rope_create(rot_dim, interleaved, self.freq, mscale)

    def close(self) -> None:
        if self.handle:
            mlora.mlora_rope_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SeqMeta:
    """One step's sequences (token rows, cached lengths, page tables) and the attention's workspace, for layers of
    n_q_heads query heads over n_kv_heads key/value heads."""

    def __init__(self, max_seqs: int, max_tokens: int, max_pages: int, n_q_heads: int, n_kv_heads: int, head_dim: int):
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.device = torch.device("cuda", torch.cuda.current_device())
        self.handle = mlora.mlora_seq_create(max_seqs, max_tokens, max_pages, n_q_heads, n_kv_heads, head_dim)
        self.T = 0
        self.n_seqs = 0

    def build(self, q_start: torch.Tensor, kv_len: torch.Tensor, pages: torch.Tensor, T: int, cache: KVCache,
              max_new: int, stream=None) -> None:
        """q_start int32 [n_seqs + 1], kv_len int32 [n_seqs], pages int32 [n_seqs, >= max_pages], all on the GPU."""
        for x in (q_start, kv_len, pages):
            assert x.is_cuda and x.dtype == torch.int32 and x.is_contiguous()
        n = kv_len.shape[0]
        assert q_start.shape == (n + 1,) and pages.dim() == 2 and pages.shape[0] == n
        mlora.mlora_build_seq(self.handle, q_start, kv_len, pages, pages.shape[1], n, T, max_new, cache.handle,
                              _raw_stream(stream, self.device))
        self.T, self.n_seqs = T, n

    def status(self) -> None:
        mlora.mlora_seq_status(self.handle)

    def close(self) -> None:
        if self.handle:
            mlora.mlora_seq_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def qkv_write(cache: KVCache, seq: SeqMeta, qkv: torch.Tensor, q: torch.Tensor | None = None, q_norm=None, k_norm=None,
              eps: float = 1e-6, rope: Rope | None = None, positions=None, stream=None) -> torch.Tensor:
    """Norm and rotation of the step's qkv rows (fp32 [T, (Hq + 2 Hkv) hd], rows may be strided); keys and values to
    the cache, queries bf16 [T, Hq, hd]."""
    hq, hkv, hd = seq.n_q_heads, seq.n_kv_heads, seq.head_dim
    assert qkv.is_cuda and qkv.dtype == torch.float32 and qkv.shape == (seq.T, (hq + 2 * hkv) * hd) and qkv.stride(1) == 1
    for x in (q_norm, k_norm):
        assert x is None or (x.is_cuda and x.dtype == torch.bfloat16 and x.shape == (hd,) and x.is_contiguous())
    assert positions is None or (positions.is_cuda and positions.dtype == torch.int32 and positions.shape == (seq.T,)
                                 and positions.is_contiguous())
    if q is None:
        q = _output((seq.T, hq, hd), torch.bfloat16, seq.device, stream)
    else:
        assert q.is_cuda and q.dtype == torch.bfloat16 and q.shape == (seq.T, hq, hd) and q.is_contiguous()
    mlora.mlora_qkv_write(cache.handle, seq.handle, qkv, qkv.stride(0) if seq.T > 1 else qkv.shape[1], q_norm, k_norm,
                          eps, rope.handle if rope is not None else None, positions, q, _raw_stream(stream, seq.device))
    return q


def attention(cache: KVCache, seq: SeqMeta, q: torch.Tensor, o: torch.Tensor | None = None, scale: float | None = None,
              stream=None) -> torch.Tensor:
    """Causal attention of the step's queries (bf16 [T, Hq, hd]) over the cache: bf16 [T, Hq * hd], the o linear's
    input. scale: 1 / sqrt(hd) by default. Over an e4m3 cache keys whose weight (or weight times value scale) is less than
    2^-21 of the row's largest count with fewer bits, below 2^-31 they may count as zero."""
    hq, hd = seq.n_q_heads, seq.head_dim
    assert q.is_cuda and q.dtype == torch.bfloat16 and q.shape == (seq.T, hq, hd) and q.is_contiguous()
    if o is None:
        o = _output((seq.T, hq * hd), torch.bfloat16, seq.device, stream)
    else:
        assert o.is_cuda and o.dtype == torch.bfloat16 and o.shape == (seq.T, hq * hd) and o.is_contiguous()
    mlora.mlora_attention(cache.handle, seq.handle, q, hd ** -0.5 if scale is None else scale, o, _raw_stream(stream, seq.device))
    return o


def kv_read(cache: KVCache, seq: SeqMeta, row_start: torch.Tensor, rows: int, k=None, v=None, stream=None) -> tuple:
    """The step's sequences as dense rows: position p of sequence s is row row_start[s] + p of k, v (bf16
    [rows, Hkv, hd]). row_start: int32, at least one entry for each sequence."""
    assert row_start.is_cuda and row_start.dtype == torch.int32 and row_start.is_contiguous()
    assert row_start.numel() >= seq.n_seqs
    shape = (rows, cache.n_kv_heads, cache.head_dim)
    if k is None:
        k = _output(shape, torch.bfloat16, seq.device, stream)
    if v is None:
        v = _output(shape, torch.bfloat16, seq.device, stream)
    assert k.is_cuda and v.is_cuda and k.shape == shape and v.shape == shape and k.dtype == v.dtype == torch.bfloat16
    assert k.is_contiguous() and v.is_contiguous()
    mlora.mlora_kv_read(cache.handle, seq.handle, row_start, rows, k, v, _raw_stream(stream, seq.device))
    return k, v


def attention_block(meta: StepMeta, seq: SeqMeta, cache: KVCache, x: torch.Tensor, qkv_pool: AdapterPool, W_qkv: torch.Tensor,
                    o_pool: AdapterPool, W_o: torch.Tensor, q_norm=None, k_norm=None, eps: float = 1e-6,
                    rope: Rope | None = None, scale: float | None = None, stream=None) -> torch.Tensor:
    """One layer's attention for the step that `meta` (adapters) and `seq` (sequences) describe: the adapted qkv linear of
    x (bf16 [T, hidden]), the write of its rows, the attention over the cache, and the adapted o linear: fp32
    [T, W_o.shape[0]]. With `stream` all of it runs there, what lies between the operators included."""
    if stream is not None:
        here = torch.cuda.current_stream(seq.device)
        with torch.cuda.stream(_torch_stream(stream, seq.device)):
            y = attention_block(meta, seq, cache, x, qkv_pool, W_qkv, o_pool, W_o, q_norm, k_norm, eps, rope, scale)
        y.record_stream(here)
        return y
    qkv = linear(qkv_pool, meta, x, W_qkv)
    q = qkv_write(cache, seq, qkv, q_norm=q_norm, k_norm=k_norm, eps=eps, rope=rope)
    return linear(o_pool, meta, attention(cache, seq, q, scale=scale), W_o)
