"""The attention step (cache write, attention, cache read) against fp64, element by element.

Tolerances, from the arithmetic:
             (Half a step of a type with b significant bits is 2^-b relative: bf16 2^-8, f16 2^-11, e4m3 2^-4.)
  attention  an output is sum_j P_j v_j / sum_j p_j rounded to bf16 (2^-8 |o|). The weights P are rounded once, to
             bf16 (2^-8) or, over an e4m3 cache, f16 (2^-11): at most that times W = sum_j p_j |v_j|. A score error d
             changes the weights by at most 2 d relative: scores are fp32 sums of hd exact products (hd 2^-24 times
             S = max_j scale sum |q k|), and over an e4m3 cache the queries are rounded to f16 (2^-11 S). The base-2
             exponential and its argument add about 2^-20 S. Weights may be summed at 2^8 of the maximum, which
             changes no relative error.
  write      bf16 results: 2^-8 relative, plus 2e-6 of the row's largest element for the norm, the angles (1e-7) and
             the rotation in fp32. e4m3: half a step, 2^-4 relative or 2^-10 of the scale, plus the same; the scale 4e-6.
  read       bf16 caches exactly; e4m3: the fp32 product rounded once, exactly."""
import numpy as np
import pytest

from oracle import attention as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layer():
    from rank_adapter_gemm_token_gb300 import layer
    return layer


class Step:
    """A step of sequences with n[s] new tokens on top of ctx[s] cached ones, in a cache full of NaN elsewhere."""

    def __init__(self, layer, n, ctx, hq=8, hkv=2, hd=128, page=16, kind="bf16", seed=0, tail=0, lead=0, spare=2,
                 n_pages=None, max_new=None, q_gain=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.layer, self.n, self.len = layer, list(n), [a + b for a, b in zip(n, ctx)]
        self.hq, self.hkv, self.hd, self.page, self.kind = hq, hkv, hd, page, kind
        used = [-(-x // page) for x in self.len]
        n_pages = n_pages or sum(used) + spare
        self.starts = [lead]
        for x in n:
            self.starts.append(self.starts[-1] + x)
        self.T = self.starts[-1] + tail
        shape = (n_pages, hkv, page, hd)
        e4m3 = kind == "e4m3"
        self.k, self.v = (torch.full(shape, 127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if e4m3 else
                          torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.ks, self.vs = ((torch.full(shape[:3], float("nan"), device="cuda") if e4m3 else None) for _ in range(2))
        perm = torch.randperm(n_pages, generator=g, device="cuda").cpu().tolist() if n_pages < 1 << 16 else list(
            range(n_pages - 1, n_pages - 1 - sum(used), -1))
        table = np.full((len(n), max(max(used), 1)), -1, dtype=np.int32)
        self.rows = []                                     # (k, v) fp64 [L, hkv, hd] of each sequence
        gain = torch.exp(torch.randn(1, hkv, hd, generator=g, device="cuda"))
        for s, L in enumerate(self.len):
            mine = [perm.pop() for _ in range(used[s])]
            table[s, :used[s]] = mine
            dense = []
            for x, z, up in ((self.k, self.ks, gain), (self.v, self.vs, 1.0)):
                a = (torch.randn(L, hkv, hd, generator=g, device="cuda") * up).to(torch.bfloat16)
                if e4m3:
                    a = a.float() * torch.exp(3 * torch.randn(L, hkv, 1, generator=g, device="cuda"))   # scales of many sizes
                    sc = a.abs().amax(-1) / 448
                    code = (a / sc[..., None]).to(torch.float8_e4m3fn)
                    dense.append((code.double() * sc.double()[..., None]).cpu().numpy())
                else:
                    dense.append(a.double().cpu().numpy())
                for i, p in enumerate(mine):
                    r = slice(i * page, min((i + 1) * page, L))
                    m = r.stop - r.start
                    if e4m3:
                        x.view(torch.uint8)[p, :, :m] = code[r].view(torch.uint8).transpose(0, 1)
                        z[p, :, :m] = sc[r].T
                    else:
                        x[p, :, :m] = a[r].transpose(0, 1)
            self.rows.append(dense)
        self.q = (torch.randn(self.T, hq, hd, generator=g, device="cuda") * q_gain).to(torch.bfloat16)
        self.q_start = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(self.len, dtype=torch.int32, device="cuda")
        self.table = torch.from_numpy(table).cuda()
        self.cache = layer.KVCache(n_pages, page, hkv, hd, k=self.k, v=self.v, k_scale=self.ks, v_scale=self.vs)
        self.seq = layer.SeqMeta(len(n), max(self.T, 1), table.shape[1], hq, hkv, hd)
        self.max_new = max(n) if max_new is None else max_new
        self.build()

    def build(self):
        self.seq.build(self.q_start, self.kv_len, self.table, self.T, self.cache, self.max_new)

    def run(self, **kw):
        o = torch.full((self.T, self.hq * self.hd), 7.0, dtype=torch.bfloat16, device="cuda")
        return self.layer.attention(self.cache, self.seq, self.q, o, **kw)

    def check(self, o, rows=None, scale=None):
        scale = self.hd ** -0.5 if scale is None else scale
        want, W, S = ref.attention(self.q.double().cpu().numpy(), [r[0] for r in self.rows], [r[1] for r in self.rows],
                                   self.starts, self.hq // self.hkv, scale)
        got = o.double().cpu().numpy().reshape(want.shape)
        up, uq = (2.0 ** -8, 0.0) if self.kind == "bf16" else (2.0 ** -11, 2.0 ** -11)
        d = (uq + self.hd * 2.0 ** -24 + 2.0 ** -20) * S[..., None]
        tol = 2.0 ** -8 * np.abs(want) + (up + 2 * d) * (W + np.abs(want)) + 1e-30
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(got - want) / tol)))


CASES = [
    # new, earlier, heads, kv heads, hd, page
    ([1], [0], 1, 1, 128, 16),                                    # one key
    ([1], [0], 8, 2, 64, 8),
    ([1, 1, 1, 1], [0, 15, 16, 17], 8, 2, 128, 16),               # around a page's end
    ([1, 1, 1], [63, 64, 130], 7, 1, 128, 64),                    # around a unit's end, an odd group
    ([1, 0, 1, 0], [40, 30, 0, 0], 8, 8, 64, 32),                 # no new tokens, an empty sequence
    ([1] * 9, [5, 300, 0, 77, 1000, 31, 32, 33, 2], 32, 8, 128, 16),
    ([1, 1], [700, 20], 16, 1, 128, 16),                          # 16 rows of one token
    ([1, 1], [700, 20], 24, 1, 128, 16),                          # 24 rows: above the row kernel's limit
    ([2, 1, 2], [0, 90, 200], 8, 2, 128, 8),                      # up to 8 rows
    ([3, 4, 1], [0, 90, 200], 8, 2, 64, 16),                      # up to 16 rows
    ([1, 5, 1, 40, 1], [100, 0, 3, 60, 17], 8, 2, 128, 16),       # single tokens beside chunks
    ([17], [0], 1, 1, 128, 16),
    ([127, 128, 129], [0, 0, 0], 2, 2, 128, 16),                  # around a tile of keys and of rows
    ([33], [95], 4, 1, 64, 8),                                    # 132 rows over 128 keys
    ([37, 0, 64], [219, 5, 64], 7, 1, 128, 256),                  # odd group, page larger than a tile
    ([100], [0], 28, 4, 64, 128),
    ([200], [57], 3, 3, 64, 32),
    ([20, 300], [900, 0], 4, 2, 128, 64),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(layer, case, kind):
    n, ctx, hq, hkv, hd, page = CASES[case]
    st = Step(layer, n, ctx, hq, hkv, hd, page, kind, seed=case)
    o = st.run()
    st.seq.status()
    st.check(o)
    again = st.run()
    assert torch.equal(o, again), "a repeated call differs"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,ctx,hq,hkv", [([1], [20000], 4, 1), ([1, 1], [9000, 3], 8, 2), ([3], [5000], 4, 1),
                                           ([9], [6000], 4, 1), ([70], [4000], 4, 2), ([5, 1, 1], [3000, 8000, 1], 8, 1)])
def test_long_axis_is_split_and_joined(layer, n, ctx, hq, hkv, kind):
    st = Step(layer, n, ctx, hq, hkv, kind=kind, page=64, seed=5)
    o = st.run()
    st.seq.status()
    st.check(o)
    for _ in range(3):
        assert torch.equal(o, st.run()), "the parts' order changes the result"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("seqs,hq,hkv,hd", [(8, 32, 8, 64), (5, 32, 8, 128), (4, 20, 4, 64), (7, 8, 8, 64)])
def test_items_of_many_parts_side_by_side(layer, seqs, hq, hkv, hd, kind):
    """A few sequences, so that each one's keys go to nine or more CTAs and most CTAs end one item and begin the next: the parts of
    neighbours are told apart, whatever their numbers, and a call leaves nothing behind for the next."""
    for k in range(6):
        ctx = [752 + 997 * (i + 1) * (k + 1) % 2259 for i in range(seqs)]
        st = Step(layer, [1] * seqs, ctx, hq, hkv, hd, 64, kind, seed=40 + k)
        o = st.run()
        st.seq.status()
        st.check(o)
        for _ in range(5):
            assert torch.equal(o, st.run())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_blocks_of_one_tile_between_others(layer, kind):
    """Prompts of 660 tokens: each one's last block has rows in its first tile alone, and its run of six key tiles is followed
    in the same CTA by the next prompt's first block, where both tiles have rows."""
    st = Step(layer, [660] * 6, [0] * 6, 32, 8, hd=64, page=64, kind=kind, seed=9)
    o = st.run()
    st.seq.status()
    st.check(o)


# Steps with more blocks of rows than there are CTAs, which the tile kernel takes whole: a few each, of very different
# lengths; many each; more than the plan keeps in shared memory.
DEALT = [
    ([700, 90, 333, 512, 61, 900, 40], [0, 300, 0, 64, 700, 0, 129], 32, 8, 128),
    ([17 + 7 * i % 44 for i in range(200)], [13 * i % 90 for i in range(200)], 8, 8, 64),
    ([1 + i % 2 for i in range(4200)], [i % 5 for i in range(4200)], 24, 1, 64),
]


# (Not the second with e4m3: its scales, spread over 2^40, leave sums to weights of 2^-54, which are zero in f16.)
@pytest.mark.parametrize("case,kind", [(0, "bf16"), (1, "bf16"), (2, "bf16"), (0, "e4m3"), (2, "e4m3")])
def test_whole_blocks_dealt_out(layer, case, kind):
    n, ctx, hq, hkv, hd = DEALT[case]
    st = Step(layer, n, ctx, hq, hkv, hd, 32, kind, seed=20 + case)
    o = st.run()
    st.seq.status()
    st.check(o)
    for _ in range(3):
        st.build()
        assert torch.equal(o, st.run()), "who takes a block changes the result"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_scores_and_rising_maxima(layer, kind):
    """Scores of tens to hundreds: the running maximum moves often, and late."""
    for n, ctx in (([1, 2], [900, 300]), ([60], [500])):
        st = Step(layer, n, ctx, 4, 1, kind=kind, seed=3, q_gain=6.0)
        o = st.run(scale=0.5)
        st.check(o, scale=0.5)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_of_no_sequence_are_zero(layer, kind):
    st = Step(layer, [1, 30, 2], [50, 20, 0], kind=kind, lead=3, tail=5)
    o = st.run()
    st.check(o)
    assert not o[:3].any() and not o[-5:].any()
    st.kv_len[1] = 0                                       # padding: a sequence without a length
    st.build()
    o = st.run()
    st.seq.status()
    assert not o[st.starts[1]:st.starts[2]].any()
    keep = st.rows[1]
    st.rows[1] = [keep[0][:0], keep[1][:0]]
    st.check(o)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_non_finite_rows_reach_their_own_sequence_alone(layer, kind):
    st = Step(layer, [1, 1, 20, 20], [40, 40, 40, 40], 4, 2, kind=kind)
    clean = st.run()
    for s in (1, 3):
        p = int(st.table[s, 1])
        if kind == "bf16":
            st.k[p, 0, 2] = float("nan")
        else:
            st.ks[p, 0, 2] = float("nan")
    o = st.run()
    a, b = st.starts[1], st.starts[3]
    half = 2 * st.hd
    assert torch.isnan(o[a, :half]).all() and torch.isnan(o[b:, :half]).all()
    assert torch.equal(o[a, half:], clean[a, half:]) and torch.equal(o[b:, half:], clean[b:, half:])
    assert torch.equal(o[0], clean[0]) and torch.equal(o[st.starts[2]:b], clean[st.starts[2]:b])


def test_zero_queries_average_the_values(layer):
    for kind in ("bf16", "e4m3"):
        st = Step(layer, [1, 40], [100, 10], 4, 1, kind=kind)
        st.q.zero_()
        st.check(st.run())


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_another_stream(layer, kind):
    st = Step(layer, [1, 40], [300, 100], kind=kind)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        st.build()
        o = st.run()
    s.synchronize()
    st.check(o)
    o2 = torch.empty_like(o)
    layer.attention(st.cache, st.seq, st.q, o2, stream=s)
    s.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_operands_aligned_to_16_bytes_alone(layer, kind):
    from rank_adapter_gemm_token_gb300 import mlora
    st = Step(layer, [1, 40, 2], [300, 100, 0], kind=kind)
    whole = st.run()
    wide = torch.empty(st.T * st.hq * st.hd + 8, dtype=torch.bfloat16, device="cuda")
    q = torch.empty_like(wide)
    q[8:] = st.q.flatten()
    mlora.mlora_attention(st.cache.handle, st.seq.handle, q.data_ptr() + 16, st.hd ** -0.5, wide.data_ptr() + 16)
    torch.cuda.synchronize()
    assert torch.equal(wide[8:].view_as(whole), whole)


def test_offsets_past_32_bits(layer):
    """A cache of 5.2e9 elements each for K and V, the sequences in its last pages."""
    st = Step(layer, [1, 20], [100, 100], 8, 8, page=16, n_pages=320000)
    assert st.k.numel() > 1 << 32 and int(st.table[0, 0]) > 319000
    o = st.run()
    st.check(o)
    k, v = layer.kv_read(st.cache, st.seq, torch.tensor([0, 101], dtype=torch.int32, device="cuda"), 221)
    assert torch.equal(k.double().cpu(), torch.from_numpy(np.concatenate([r[0] for r in st.rows])))
    assert torch.equal(v.double().cpu(), torch.from_numpy(np.concatenate([r[1] for r in st.rows])))
    qkv = torch.randn(21, 24 * 128, device="cuda")
    layer.qkv_write(st.cache, st.seq, qkv)
    p, off = int(st.table[0, 100 // 16]), 100 % 16
    assert torch.equal(st.k[p, :, off], qkv[0, 1024:2048].view(8, 128).to(torch.bfloat16))


def test_graph_replay_follows_the_arrays(layer):
    st = Step(layer, [1, 30], [200, 40])
    out = torch.empty(st.T, st.hq * st.hd, dtype=torch.bfloat16, device="cuda")
    run = lambda: (st.build(), layer.attention(st.cache, st.seq, st.q, out))  # noqa: E731
    run()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    st.kv_len[0] = 120
    st.rows[0] = [r[:120] for r in st.rows[0]]
    g.replay()
    torch.cuda.synchronize()
    st.check(out)


# ------------------------------------------------------------------------------------------- refusals
def test_rejected_sequences_are_skipped_and_named(layer):
    from rank_adapter_gemm_token_gb300 import mlora

    def spoil(what):
        st = Step(layer, [1, 30, 1], [50, 20, 10])
        bad = 1
        if what == "page":
            st.table[1, 2] = st.k.shape[0]
        elif what == "negative page":
            st.table[1, 0] = -1
        elif what == "length":
            st.kv_len[1] = 29
        elif what == "long":
            st.kv_len[1] = st.table.shape[1] * st.page + 1
        elif what == "negative length":
            st.kv_len[1] = -5
        elif what == "more than max_new":
            st.max_new = 29
        elif what == "descending":
            st.q_start[1], bad = 40, 0
        elif what == "beyond T":
            st.q_start[3], bad = 40, 2
        elif what == "overlapping":
            st.q_start.copy_(torch.tensor([0, 30, 2, 32], dtype=torch.int32))
            st.max_new = 32
        st.build()
        o = st.run()
        with pytest.raises(mlora.MloraError) as e:
            st.seq.status()
        assert e.value.status == mlora.MLORA_ERR_BAD_SEQUENCE, what
        st.seq.status()                                   # reported once
        return st, o, bad, str(e.value)

    for what in ("page", "negative page", "length", "long", "negative length", "more than max_new"):
        st, o, bad, text = spoil(what)
        assert "sequence 1" in text
        assert not o[1:31].any(), what
        st.rows[1] = [r[:0] for r in st.rows[1]]
        st.check(o)
        row = st.layer.qkv_write(st.cache, st.seq, torch.randn(st.T, 12 * 128, device="cuda"))
        assert not row[1:31].any() and row[0].any()
    for what in ("descending", "beyond T", "overlapping"):
        spoil(what)


def test_arguments_are_refused(layer):
    from rank_adapter_gemm_token_gb300 import mlora as m
    st = Step(layer, [1, 30], [50, 20])
    other = layer.KVCache(4, 32, 2, 128)
    wide = layer.KVCache(st.k.shape[0], 16, 4, 128)
    q, o, seq, kv = st.q, torch.empty_like(st.q), st.seq.handle, st.cache.handle
    qkv = torch.zeros(st.T, 12 * 128, device="cuda")
    long_rope = layer.Rope(128)
    small = Step(layer, [1], [3], hd=64)

    def status(call, *a):
        with pytest.raises(m.MloraError) as e:
            call(*a)
        return e.value.status

    fresh = m.mlora_seq_create(2, 8, 2, 8, 2, 128)
    assert status(m.mlora_attention, kv, fresh, q, 1.0, o) == m.MLORA_ERR_INVALID_ARG                 # not built
    assert status(m.mlora_attention, other.handle, seq, q, 1.0, o) == m.MLORA_ERR_MISMATCH             # other pages
    assert status(m.mlora_attention, wide.handle, seq, q, 1.0, o) == m.MLORA_ERR_MISMATCH              # other heads
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert status(m.mlora_attention, kv, seq, q, scale, o) == m.MLORA_ERR_INVALID_ARG
    assert status(m.mlora_attention, kv, seq, None, 1.0, o) == m.MLORA_ERR_INVALID_ARG
    assert status(m.mlora_attention, kv, seq, q.data_ptr() + 2, 1.0, o) == m.MLORA_ERR_INVALID_ARG
    for a in ((qkv, 12 * 128 - 4, None, None, 0.0, None, None, q), (qkv, 12 * 128 + 2, None, None, 0.0, None, None, q),
              (None, 12 * 128, None, None, 0.0, None, None, q), (qkv, 12 * 128, None, None, 0.0, None, None, None),
              (qkv.data_ptr() + 4, 12 * 128, None, None, 0.0, None, None, q), (qkv, 12 * 128, q, q, -1.0, None, None, q)):
        assert status(m.mlora_qkv_write, kv, seq, *a) == m.MLORA_ERR_INVALID_ARG
    assert status(m.mlora_qkv_write, small.cache.handle, small.seq.handle, torch.zeros(1, 12 * 64, device="cuda"), 12 * 64,
                  None, None, 0.0, long_rope.handle, None, torch.empty(1, 8, 64, dtype=torch.bfloat16, device="cuda")) == m.MLORA_ERR_MISMATCH
    assert status(m.mlora_kv_read, kv, seq, None, 4, q, o) == m.MLORA_ERR_INVALID_ARG
    assert status(m.mlora_kv_read, kv, seq, st.q_start, -1, q, o) == m.MLORA_ERR_INVALID_ARG
    args = (st.q_start, st.kv_len, st.table, st.table.shape[1])
    assert status(m.mlora_build_seq, seq, *args, 3, 31, 30, kv) == m.MLORA_ERR_TOO_MANY_TOKENS
    assert status(m.mlora_build_seq, seq, *args, 2, 32, 30, kv) == m.MLORA_ERR_TOO_MANY_TOKENS
    assert status(m.mlora_build_seq, seq, *args, 2, -1, 30, kv) == m.MLORA_ERR_INVALID_ARG
    assert status(m.mlora_build_seq, seq, *args[:3], 1, 2, 31, 30, kv) == m.MLORA_ERR_INVALID_ARG       # short table rows
    assert status(m.mlora_build_seq, seq, *args, 2, 31, 30, wide.handle) == m.MLORA_ERR_MISMATCH
    m.mlora_seq_destroy(fresh)


def test_empty_steps(layer):
    st = Step(layer, [1, 30], [50, 20])
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    for T in (0, 7):                                       # no sequences, with and without rows
        st.seq.build(none, none[:0], st.table[:0], T, st.cache, 0)
        o = torch.ones(T, st.hq * st.hd, dtype=torch.bfloat16, device="cuda")
        layer.attention(st.cache, st.seq, st.q[:T], o)
        assert not o.any()
        q = layer.qkv_write(st.cache, st.seq, torch.ones(T, 12 * 128, device="cuda"))
        assert not q.any()
        layer.kv_read(st.cache, st.seq, none[:0], 0)
        st.seq.status()
    st.build()
    st.check(st.run())


# ------------------------------------------------------------------------------------------- write
def written(st, q, qkv, q_norm, k_norm, eps, rope, positions=None):
    """Checks q_out and the cache rows of the step's tokens against fp64."""
    hq, hkv, hd = st.hq, st.hkv, st.hd
    x = qkv.double().cpu().numpy().reshape(st.T, hq + 2 * hkv, hd)
    xq, xk, xv = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if q_norm is not None:
        xq = ref.norm_heads(xq, q_norm.double().cpu().numpy(), eps)
    if k_norm is not None:
        xk = ref.norm_heads(xk, k_norm.double().cpu().numpy(), eps)
    pos = np.zeros(st.T)
    for s, L in enumerate(st.len):
        a, b = st.starts[s], st.starts[s + 1]
        pos[a:b] = np.arange(L - (b - a), L)
    turn = pos if positions is None else positions.cpu().numpy().astype(np.float64)
    if rope is not None:
        xq, xk = (ref.rotate(y, turn, rope.freq, rope.interleaved, rope.mscale) for y in (xq, xk))
    inside = np.zeros(st.T, bool)
    inside[st.starts[0]:st.starts[-1]] = True
    got = q.double().cpu().numpy()
    big = np.abs(xq).max(-1, keepdims=True)
    assert (np.abs(got - xq) <= 2.0 ** -8 * np.abs(xq) + 2e-6 * big)[inside].all()
    assert not got[~inside].any()
    k, v = st.k.double().cpu().numpy(), st.v.double().cpu().numpy()
    table = st.table.cpu().numpy()
    for s in range(len(st.len)):
        for t in range(st.starts[s], st.starts[s + 1]):
            p, off = table[s, int(pos[t]) // st.page], int(pos[t]) % st.page
            for cache, scales, want in ((k, st.ks, xk[t]), (v, st.vs, xv[t])):
                row, top = cache[p, :, off], np.abs(want).max(-1, keepdims=True)
                if st.kind == "bf16":
                    assert (np.abs(row - want) <= 2.0 ** -8 * np.abs(want) + 2e-6 * top).all()
                else:
                    sc = scales[p, :, off].double().cpu().numpy()
                    exact = ref.row_scale(want)
                    assert (np.abs(sc - exact) <= 4e-6 * exact).all()
                    assert (np.abs(row * sc[:, None] - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * sc[:, None] + 1e-5 * top).all()


WRITES = [
    # new, earlier, hq, hkv, hd, page, norm, rot, interleaved, mscale
    ([1], [0], 1, 1, 128, 16, True, 128, False, 1.0),
    ([1, 1, 1], [15, 16, 700], 8, 2, 128, 16, True, 128, False, 1.0),
    ([5, 0, 40], [3, 9, 100], 7, 1, 64, 8, False, 64, True, 1.2),
    ([5, 0, 40], [3, 9, 100], 32, 8, 128, 32, False, 24, False, 1.0),
    ([300], [70], 12, 12, 64, 64, True, 24, True, 1.0),
    ([600, 1], [0, 90000], 32, 8, 128, 256, True, 64, False, 0.7),
    ([20], [11], 8, 8, 128, 16, False, 0, False, 1.0),
    ([2], [1000000], 4, 1, 128, 256, False, 128, True, 1.0),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_qkv_write(layer, case, kind):
    n, ctx, hq, hkv, hd, page, norm, rot, inter, mscale = WRITES[case]
    st = Step(layer, n, ctx, hq, hkv, hd, page, kind, seed=case, lead=2, tail=3)
    g = torch.Generator(device="cuda").manual_seed(case)
    wide = torch.randn(st.T, (hq + 2 * hkv) * hd + 8, generator=g, device="cuda") * 3
    qkv = wide[:, :-8]                                      # strided rows
    w = [(1 + 0.2 * torch.randn(hd, generator=g, device="cuda")).to(torch.bfloat16) if norm else None for _ in range(2)]
    rope = layer.Rope(rot, 10000.0, inter, mscale=mscale) if rot else None
    before = [x.view(torch.uint8).clone() for x in (st.k, st.v)]
    q = layer.qkv_write(st.cache, st.seq, qkv, q_norm=w[0], k_norm=w[1], eps=1e-5, rope=rope)
    st.seq.status()
    written(st, q, qkv, w[0], w[1], 1e-5, rope)
    if len(st.len) and max(st.len) < 2000:                  # nothing else in the cache has changed
        touched = torch.zeros(st.k.shape[0], st.page, dtype=torch.bool)
        for s, L in enumerate(st.len):
            for p in range(L - st.n[s], L):
                touched[int(st.table[s, p // page]), p % page] = True
        for x, old in zip((st.k, st.v), before):
            same = (x.view(torch.uint8) == old).all(-1).all(1).cpu()
            assert same[~touched].all()


def test_positions_and_one_norm(layer):
    st = Step(layer, [6, 1], [10, 33])
    qkv = torch.randn(st.T, 12 * 128, device="cuda")
    w = (1 + 0.2 * torch.randn(128, device="cuda")).to(torch.bfloat16)
    rope = layer.Rope(128, 500000.0)
    positions = torch.tensor([5, 0, 70000, 3, -2, 9, 1 << 20], dtype=torch.int32, device="cuda")
    q = layer.qkv_write(st.cache, st.seq, qkv, k_norm=w, eps=1e-6, rope=rope, positions=positions)
    written(st, q, qkv, None, w, 1e-6, rope, positions)


def test_e4m3_rows_at_the_edges(layer):
    st = Step(layer, [6], [0], 1, 1, kind="e4m3")
    qkv = torch.randn(6, 3 * 128, device="cuda")
    qkv[0, 128:256] = 0                                     # a zero row
    qkv[1, 128:256] *= 1e30
    qkv[2, 128:256] *= 2.0 ** -100                          # below the smallest scale's row
    qkv[3, 130] = float("inf")
    qkv[4, 140] = float("nan")
    qkv[5, 128:256] = 0
    qkv[5, 200] = -1.0
    layer.qkv_write(st.cache, st.seq, qkv)
    p = int(st.table[0, 0])
    code, sc = st.k[p, 0, :6].float(), st.ks[p, 0, :6]
    least = float(np.float32(2.0 ** -60) / np.float32(448.0))
    assert not code[0].any() and float(sc[0]) == least and float(sc[2]) == least
    assert torch.isnan(sc[3]) and torch.isnan(sc[4]) and not code[3].any() and not code[4].any()
    assert torch.allclose(code[1] * sc[1], qkv[1, 128:256], rtol=2 ** -4, atol=float(sc[1]) * 2 ** -9)
    assert float(code[5, 72]) == -448.0 and float(sc[5]) == float(np.float32(1.0) / np.float32(448.0))
    k, v = layer.kv_read(st.cache, st.seq, torch.zeros(1, dtype=torch.int32, device="cuda"), 6)
    assert torch.isnan(k[3]).all() and torch.isnan(k[4]).all() and torch.isfinite(k[[0, 1, 2, 5]]).all() and torch.isfinite(v).all()


# ------------------------------------------------------------------------------------------- read
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx,hkv,hd,page", [([0], 1, 128, 16), ([15, 16, 0, 100], 2, 64, 16), ([7, 250], 3, 128, 8),
                                             ([1000, 1, 300], 8, 128, 256), ([33] * 40, 2, 64, 32)])
def test_kv_read(layer, ctx, hkv, hd, page, kind):
    st = Step(layer, [1] * len(ctx), ctx, hkv * 2, hkv, hd, page, kind)
    gap = 3                                                 # rows between the sequences stay as they are
    start, at = [], 0
    for L in st.len:
        start.append(at)
        at += L + gap
    rs = torch.tensor(start, dtype=torch.int32, device="cuda")
    k, v = (torch.full((at, hkv, hd), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.kv_read(st.cache, st.seq, rs, at, k, v)
    st.seq.status()
    for s, L in enumerate(st.len):
        for out, dense in ((k, st.rows[s][0]), (v, st.rows[s][1])):
            want = torch.from_numpy(dense).float().to(torch.bfloat16) if kind == "bf16" else None
            got = out[start[s]:start[s] + L].cpu()
            if kind == "e4m3":                              # the product in fp32, then rounded once
                want = torch.from_numpy(dense.astype(np.float32)).to(torch.bfloat16)
            assert torch.equal(got, want)
            assert (out[start[s] + L:start[s] + L + gap] == 7.0).all()


def test_kv_read_outside_its_rows_is_reported(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    st = Step(layer, [1, 1], [20, 30])
    for rs, rows in (([0, 21], 51), ([-1, 21], 60)):
        k, v = (torch.full((rows + 8, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mlora.mlora_kv_read(st.cache.handle, st.seq.handle, torch.tensor(rs, dtype=torch.int32, device="cuda"), rows, k, v)
        with pytest.raises(mlora.MloraError) as e:
            st.seq.status()
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
        assert (k[rows:] == 7.0).all() and (v[rows:] == 7.0).all()


# ------------------------------------------------------------------------------------------- the layer
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_example_stepwise_equals_one_step(kind):
    """The same keys and values are cached either way; queries and outputs differ by bf16 rounding (2^-8 a value at most, in
    three places) and, e4m3, by codes that a last-bit difference of the linear's sums moves to the neighbour (rare)."""
    from examples import attention_serving
    assert attention_serving.main(kind) <= 3 * 2.0 ** -8


def test_attention_block_against_fp64(layer):
    """The adapted layer in fp64. Rounding to bf16 in five places (queries, keys, values, weights, the attention's output),
    each 2^-8 relative at most and about 2^-9 in the 2-norm; scores of a few units pass those of queries and keys on: 8
    roundings of 2^-9 in all."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    hidden, hq, hkv, hd, page = 512, 8, 2, 64, 16
    n, ctx = [40, 1, 1, 7], [0, 30, 100, 12]
    T, lens = sum(n), [a + b for a, b in zip(n, ctx)]
    W_qkv, W_o = rand((hq + 2 * hkv) * hd, hidden, std=0.04), rand(hidden, hq * hd, std=0.04)
    pools = layer.AdapterPool(2, 8, hidden, W_qkv.shape[0]), layer.AdapterPool(2, 8, hq * hd, hidden)
    ab = [[(rand(8, p.K, std=0.05), rand(p.D, 8, std=0.05)) for _ in range(2)] for p in pools]
    for p, mats in zip(pools, ab):
        for slot, (A, B) in enumerate(mats):
            p.load(slot, A, B, 8, 16.0)
        p.sync()
    x, slots = rand(T, hidden), torch.tensor([0] * 40 + [1, -1, 0, 1, 0, 1, 0, 1, -1], dtype=torch.int32)[:T]
    starts = np.concatenate([[0], np.cumsum(n)]).tolist()
    cache = layer.KVCache(40, page, hkv, hd)
    table = torch.arange(40, dtype=torch.int32).reshape(4, 10).cuda()
    old = [(rand(c, hkv, hd), rand(c, hkv, hd)) for c in ctx]              # what earlier steps cached
    for s, (k, v) in enumerate(old):
        for p in range(ctx[s]):
            cache.k[int(table[s, p // page]), :, p % page] = k[p]
            cache.v[int(table[s, p // page]), :, p % page] = v[p]
    meta, seq = layer.StepMeta(T, 1, 8), layer.SeqMeta(4, T, 10, hq, hkv, hd)
    meta.build(slots.cuda(), None, pools[0])
    seq.build(torch.tensor(starts, dtype=torch.int32).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table, T, cache, max(n))
    rope = layer.Rope(hd, 10000.0)
    y = layer.attention_block(meta, seq, cache, x, pools[0], W_qkv, pools[1], W_o, rope=rope)
    seq.status()
    d = lambda t: t.double().cpu().numpy()  # noqa: E731

    def linear(z, W, mats):
        out = z @ d(W).T
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                out[t] += 2.0 * d(mats[s][1]) @ (d(mats[s][0]) @ z[t])
        return out

    rows = linear(d(x), W_qkv, ab[0]).reshape(T, hq + 2 * hkv, hd)
    pos = np.concatenate([np.arange(c, c + m) for c, m in zip(ctx, n)])
    q, k = ref.rotate(rows[:, :hq], pos, rope.freq, False), ref.rotate(rows[:, hq:hq + hkv], pos, rope.freq, False)
    keys = [np.concatenate([d(o[0]), k[a:b]]) for o, a, b in zip(old, starts, starts[1:])]
    values = [np.concatenate([d(o[1]), rows[a:b, hq + hkv:]]) for o, a, b in zip(old, starts, starts[1:])]
    att, _, _ = ref.attention(q, keys, values, starts, hq // hkv, hd ** -0.5)
    want = linear(att.reshape(T, hq * hd), W_o, ab[1])
    err = np.linalg.norm(d(y) - want) / np.linalg.norm(want)
    assert err <= 8 * 2.0 ** -9, err
    for p in pools:
        p.close()
