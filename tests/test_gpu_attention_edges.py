"""The attention step at its edges: steps whose sequences do not hold, degenerate scales and scores, other streams.
Tolerances are those of test_gpu_attention.py unless a test derives its own."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_attention import Step  # noqa: E402


@pytest.fixture(scope="module")
def layer():
    from rank_adapter_gemm_token_gb300 import layer
    return layer


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------- starts that fall
def falling_step(layer, starts, T, hq, hkv, hd):
    """A step of one-page sequences (length 8, page s for sequence s) with the given starts; returns what the operators make
    of it: queries written, cache before and after, attention, rows read back, and which sequences must be served."""
    from rank_adapter_gemm_token_gb300 import mlora
    S = len(starts) - 1
    g = torch.Generator(device="cuda").manual_seed(S)
    n = [b - a for a, b in zip(starts, starts[1:])]
    most = np.maximum.accumulate(starts)
    good = [s for s in range(S) if starts[s] == most[s] and 0 <= n[s] <= 8 and starts[s + 1] <= T]
    cache = layer.KVCache(S, 8, hkv, hd)
    cache.k.normal_(generator=g)
    cache.v.normal_(generator=g)
    seq = layer.SeqMeta(S, T, 1, hq, hkv, hd)
    seq.build(ints(starts), ints([8] * S), torch.arange(S, dtype=torch.int32, device="cuda")[:, None].contiguous(), T, cache, 8)
    with pytest.raises(mlora.MloraError) as e:
        seq.status()
    assert e.value.status == mlora.MLORA_ERR_BAD_SEQUENCE
    first = next(s for s in range(S) if s not in set(good))
    assert f"sequence {first}:" in str(e.value)
    return cache, seq, good, n, g


@pytest.mark.parametrize("hq,hkv,hd", [(4, 2, 64), (32, 1, 64)])   # the row kernel, the tile kernel
@pytest.mark.parametrize("S,T,starts", [
    (4, 14, [0, 6, 2, 8, 14]),                                    # the third would share the first one's tokens
    (2500, 1, [i % 2 for i in range(2501)]),                      # one token, named by 1250 sequences
    (3000, 2100, [min(i, 1500) if i <= 1500 else 700 + (i - 1501) % 800 if i < 2400 else 1500 + i - 2400 for i in range(3001)]),
])
def test_sequences_that_start_below_an_earlier_one_are_skipped(layer, S, T, starts, hq, hkv, hd):
    assert len(starts) == S + 1
    cache, seq, good, n, g = falling_step(layer, starts, T, hq, hkv, hd)
    assert 0 < len(good) < S
    # the cache: new rows of the served sequences alone
    k0, v0 = cache.k.clone(), cache.v.clone()
    qkv = torch.randn(T, (hq + 2 * hkv) * hd, generator=g, device="cuda")
    q = layer.qkv_write(cache, seq, qkv)
    want_q = torch.zeros_like(q)
    rows = qkv.view(T, hq + 2 * hkv, hd).to(torch.bfloat16)
    for s in good:
        a, b = starts[s], starts[s + 1]
        want_q[a:b] = rows[a:b, :hq]
        k0[s, :, 8 - n[s]:] = rows[a:b, hq:hq + hkv].transpose(0, 1)
        v0[s, :, 8 - n[s]:] = rows[a:b, hq + hkv:].transpose(0, 1)
    assert torch.equal(q, want_q) and torch.equal(cache.k, k0) and torch.equal(cache.v, v0)
    # the attention: their rows, and zeros
    o = layer.attention(cache, seq, q, torch.full((T, hq * hd), 7.0, dtype=torch.bfloat16, device="cuda"))
    want, tol = torch.zeros(T, hq, hd, dtype=torch.float64, device="cuda"), torch.zeros(T, hq, hd, dtype=torch.float64, device="cuda")
    for s in good:
        a, b = starts[s], starts[s + 1]
        if a == b:
            continue
        k, v = (x[s].double().repeat_interleave(hq // hkv, 0) for x in (cache.k, cache.v))       # [hq, 8, hd]
        z = torch.einsum("thd,hjd->thj", q[a:b].double(), k) * hd ** -0.5
        hidden = torch.arange(8, device="cuda")[None] > torch.arange(8 - n[s], 8, device="cuda")[:, None]
        p = torch.softmax(z.masked_fill(hidden[:, None], float("-inf")), -1)
        want[a:b] = torch.einsum("thj,hjd->thd", p, v)
        # weights and the output rounded to bf16, scores (below 64) to 5e-6 of their size
        tol[a:b] = 2.0 ** -8 * want[a:b].abs() + (2.0 ** -8 + 1e-3) * torch.einsum("thj,hjd->thd", p, v.abs()) + 1e-30
    assert bool(((o.double().view(T, hq, hd) - want).abs() <= tol).all())
    # the cache read: their rows, in their places
    at, start = 0, []
    for s in range(S):
        start.append(at)
        at += 8 if s in set(good) else 0
    out = [torch.full((S * 8, hkv, hd), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    layer.kv_read(cache, seq, ints(start), S * 8, *out)
    seq.status()
    for x, dense in zip((cache.k, cache.v), out):
        assert torch.equal(dense[:at], x[good].transpose(1, 2).reshape(at, hkv, hd))
        assert bool((dense[at:] == 7.0).all())


def test_length_near_2_31_is_rejected(layer):
    """Rounded up to whole pages it would pass 2^31; the table has room for it."""
    from rank_adapter_gemm_token_gb300 import mlora
    cache = layer.KVCache(2, 256, 1, 64)
    seq = layer.SeqMeta(2, 2, 1 << 23, 2, 1, 64)
    table = torch.full((2, 1 << 23), 5, dtype=torch.int32, device="cuda")          # pages that are not there
    table[1, 0] = 1
    cache.v[1, 0, :3] = 2.0
    for L in (2 ** 31 - 1, 2 ** 31 - 255):
        seq.build(ints([0, 1, 2]), ints([L, 3]), table, 2, cache, 1)
        o = layer.attention(cache, seq, torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda"))
        with pytest.raises(mlora.MloraError) as e:
            seq.status()
        assert e.value.status == mlora.MLORA_ERR_BAD_SEQUENCE and "sequence 0:" in str(e.value)
        assert not o[0].any() and bool((o[1] == 2.0).all())


# ------------------------------------------------------------------------------------------- scales of an e4m3 cache
def set_scale(st, s, pos, which, value):
    """The scale of position pos of sequence s (all heads) in the cache and in the step's fp64 rows."""
    p, off = int(st.table[s, pos // st.page]), pos % st.page
    z = (st.ks, st.vs)[which]
    dense = st.rows[s][which]
    old = z[p, :, off].double().cpu().numpy()[:, None]
    z[p, :, off] = value
    dense[pos] = dense[pos] / old * float(np.float32(value))


@pytest.mark.parametrize("hq,hkv,hd", [(8, 2, 128), (8, 2, 64), (16, 1, 128)])
def test_value_scales_of_zero_keep_their_weights(layer, hq, hkv, hd):
    """Single tokens, short chunks and chunks over caches where a third of the value rows, all of them, and the whole first
    part have scale 0 (or one so small that it counts as 0): their weights stay in the denominator."""
    rng = np.random.default_rng(3)
    for n in ([1, 1, 1], [2, 1, 2], [40, 1, 30]):
        st = Step(layer, n, [300, 90, 700], hq, hkv, hd, 16, "e4m3", seed=7)
        for s, L in enumerate(st.len):
            zero = {0: rng.random(L) < 1 / 3, 1: np.ones(L, bool), 2: np.arange(L) < L // 2}[s]
            for pos in np.flatnonzero(zero):
                set_scale(st, s, int(pos), 1, 0.0 if pos % 2 else 2.0 ** -110)
        o = st.run()
        st.seq.status()
        st.check(o)
        assert not o[st.starts[1]:st.starts[2]].any()
        assert torch.equal(o, st.run())


@pytest.mark.parametrize("n", [1, 33])
def test_two_equal_scores_one_value_scale_zero(layer, n):
    """Scores of 0, codes of 448, value scales 1/448 and 0 in turn: the mean of ones and zeros."""
    st = Step(layer, [n], [64 - n], 4, 1, kind="e4m3")
    st.q.zero_()
    for pos in range(64):
        p, off = int(st.table[0, pos // 16]), pos % 16
        st.v.view(torch.uint8)[p, :, off] = 0x7E
        st.vs[p, :, off] = 1 / 448 if pos % 2 else 0.0
    o = st.run().float()
    seen = torch.arange(64 - n + 1, 65, device="cuda")
    want = (seen // 2).float() / seen
    assert bool(((o - want[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -11) * want[:, None]).all())


def test_value_scales_from_tiny_to_large(layer):
    """Scales of 2^-90 ... 2^40 among the keys of single tokens: each row's sum is that of its largest products."""
    st = Step(layer, [1, 2], [500, 60], 8, 2, kind="e4m3", seed=2, q_gain=0.2)
    rng = np.random.default_rng(5)
    for s, L in enumerate(st.len):
        for pos in range(L):
            set_scale(st, s, pos, 1, 2.0 ** rng.integers(-90, 41))
    st.check(st.run())


# ------------------------------------------------------------------------------------------- degenerate scores
@pytest.mark.parametrize("hq,hkv,n", [(4, 2, 1), (4, 2, 2), (4, 1, 60), (2, 2, 200)])
def test_rows_whose_scores_are_all_minus_infinity_are_nan(layer, hq, hkv, n):
    """A key with an infinity gives a score of -inf to queries of the other sign there: nothing, beside others; alone, 0 / 0.
    Keys 0 and 1 of kv head 0 have it; the first new token sees key 0 (and 1, for single tokens) alone."""
    st = Step(layer, [n], [1 if n == 1 else 0], hq, hkv, 128)
    st.q[:, :, 0] = -1.0
    inf = [0, 1] if n == 1 else [0]
    for pos in inf:
        st.k[int(st.table[0, 0]), 0, pos, 0] = float("inf")
    o = st.run()
    st.seq.status()
    g = hq // hkv * st.hd
    assert torch.isnan(o[0, :g]).all()
    assert torch.isfinite(o[1:]).all() and torch.isfinite(o[0, g:]).all()
    if n > 1:                                             # elsewhere the key counts nothing
        keep = st.rows[0][0]
        keep[0, 0, :] = 0.0
        st.rows[0][0] = keep
        want, W, S = attend_without(st, 0, 0)
        got = o.double().cpu().numpy().reshape(want.shape)[1:]
        d = (st.hd * 2.0 ** -24 + 2.0 ** -20) * S[..., None]
        assert (np.abs(got - want[1:]) <= (2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2 * d) * (W + np.abs(want)) + 1e-30)[1:]).all()


def attend_without(st, head, pos):
    """The step's only sequence in fp64, key `pos` left out for kv head `head`."""
    from oracle import attention as ref
    k, v = st.rows[0]
    q = st.q.double().cpu().numpy()
    G = st.hq // st.hkv
    out, W, S = ref.attention(q, [k], [v], st.starts, G, st.hd ** -0.5)
    L, n = len(k), st.n[0]
    for t in range(n):
        seen = L - n + t + 1
        keys = [j for j in range(seen) if j != pos]
        if not keys:
            continue
        for h in range(head * G, head * G + G):
            z = st.hd ** -0.5 * (k[keys, head] @ q[t, h])
            p = np.exp(z - z.max())
            p /= p.sum()
            out[t, h], W[t, h] = p @ v[keys, head], p @ np.abs(v[keys, head])
    return out, W, S


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,ctx", [(1, 20000), (9, 6000)])
def test_a_part_of_nan_alone_is_not_lost(layer, n, ctx, kind):
    """A long axis in parts, all keys from one on NaN: wherever a part begins with it, the joined rows are NaN."""
    st = Step(layer, [n], [ctx], 4, 1, 64, 64, kind, seed=6)
    assert torch.isfinite(st.run()).all()
    for i in range((ctx + n - 1) // 64, -1, -1):
        (st.k if kind == "bf16" else st.ks)[int(st.table[0, i])] = float("nan")
        seen = min(n, max(0, 64 * i - ctx))               # new tokens before key 64 i
        o = st.run()
        assert torch.isnan(o[seen:]).all() and torch.isfinite(o[:seen]).all(), i


@pytest.mark.parametrize("n", [[1, 1], [3], [50, 20]])
@pytest.mark.parametrize("hd", [64, 128])
def test_tiny_queries_over_e4m3(layer, n, hd):
    """Queries of subnormal bf16 numbers, of which f16 cannot hold the inverse of the largest, and of the largest magnitudes."""
    for gain in (2.0 ** -132, 2.0 ** -127, 2.0 ** -20, 2.0 ** 100):
        st = Step(layer, n, [70] * len(n), 4, 2, hd, kind="e4m3", seed=4)
        st.q = (st.q.double() * gain).to(torch.bfloat16)
        scale = 0.1 if gain < 1 else 0.1 / gain
        st.check(st.run(scale=scale), scale=scale)


@pytest.mark.parametrize("n,hq,hkv,hd", [([1, 1, 1], 8, 2, 128), ([1, 2], 8, 2, 64), ([4, 3], 4, 1, 128), ([150], 4, 2, 128), ([90, 40], 2, 1, 64)])
def test_sharp_scores_over_e4m3(layer, n, hq, hkv, hd):
    """Queries along one key each, with scores of 30 to 60 there: relative errors of scores show whole. Scores are fp32 sums of exact
    products (queries, lifted by a power of two, and codes times at most 7 bits of their scale are f16 numbers), times what is left of
    the scale to 2^-16; weights take what is left of the value's scale to 2^-14 and are rounded once to f16, 2^-11, and below
    2^-24 of the largest to 2^-35 of it."""
    from oracle import attention as ref
    st = Step(layer, n, [200] * len(n), hq, hkv, hd, 16, "e4m3", seed=11)
    rng = np.random.default_rng(8)
    for s, L in enumerate(st.len):
        for pos in range(L):
            for which in (0, 1):
                set_scale(st, s, pos, which, float(2.0 ** rng.uniform(-8.0, -6.0)))
    G = hq // hkv
    q = torch.zeros_like(st.q)
    for s in range(len(n)):
        for i in range(n[s]):
            for h in range(hq):
                pos = int(rng.integers(0, st.len[s] - n[s] + i + 1))
                key = st.rows[s][0][pos, h // G]
                q[st.starts[s] + i, h] = torch.from_numpy(key * rng.uniform(30, 60) / (key @ key * hd ** -0.5)).to(torch.bfloat16)
    st.q = q
    o = st.run()
    st.seq.status()
    want, W, S = ref.attention(q.double().cpu().numpy(), [r[0] for r in st.rows], [r[1] for r in st.rows], st.starts, G, hd ** -0.5)
    got = o.double().cpu().numpy().reshape(want.shape)
    d = (hd * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -16) * S[..., None]
    lost = np.zeros_like(want)
    for s in range(len(n)):
        a, b = st.starts[s], st.starts[s + 1]
        lost[a:b] = 2.0 ** -35 * 4 * np.repeat(np.abs(st.rows[s][1]).sum(0), G, 0)      # (weight times scale: scales differ by 4)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -14 + 2 * d) * (W + np.abs(want)) + lost
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(np.abs(got - want) / tol)))


@pytest.mark.parametrize("n", [1, 2, 40])
@pytest.mark.parametrize("ratio", [2.0 ** -20.37, 2.0 ** -15.6])
def test_small_weights_over_e4m3_keep_their_bits(layer, n, ratio):
    """Key 0 has nearly all of the weight and no value in the upper half of the head, where the others, of weight `ratio` each,
    have ones: weights down to 2^-21 of the largest are rounded to f16 like the others (2^-11)."""
    L = 64
    st = Step(layer, [n], [L - n], 4, 1, kind="e4m3")
    st.q.zero_()
    st.q[..., 0] = 1.0
    p = [int(st.table[0, i]) for i in range(L // 16)]
    for c, z in ((st.k, st.ks), (st.v, st.vs)):
        c.view(torch.uint8)[p] = 0
        z[p] = 1 / 448
    st.k.view(torch.uint8)[p[0], 0, 0, 0] = 0x7E          # 448: one, with its scale
    st.v.view(torch.uint8)[p, 0, :, 64:] = 0x7E
    st.v.view(torch.uint8)[p[0], 0, 0, 64:] = 0
    o = st.run(scale=-float(np.log(ratio))).double().cpu().numpy().reshape(n, 4, 128)
    others = np.arange(L - n, L)[:, None, None] * ratio
    want = np.broadcast_to(others / (1 + others), (n, 4, 64))
    # the product's one at 448 / 448 (2^-23 of a score of 20), the output's bf16 beside the weights
    assert (np.abs(o[..., 64:] - want) <= (2.0 ** -8 + 2.0 ** -11 + 1e-4) * want).all()
    assert not o[..., :64].any()


# ------------------------------------------------------------------------------------------- another stream
def busy(stream, milliseconds=100):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(2e6 * milliseconds))


class Block:
    """A small adapted layer and a step of prompts and single tokens for it."""

    def __init__(self, layer):
        g = torch.Generator(device="cuda").manual_seed(4)
        rand = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
        hidden, self.hq, self.hkv, self.hd = 512, 8, 2, 64
        self.layer = layer
        self.W_qkv, self.W_o = rand((self.hq + 2 * self.hkv) * self.hd, hidden, std=0.04), rand(hidden, self.hq * self.hd, std=0.04)
        self.pools = layer.AdapterPool(2, 8, hidden, self.W_qkv.shape[0]), layer.AdapterPool(2, 8, self.hq * self.hd, hidden)
        for p in self.pools:
            p.load(0, rand(8, p.K, std=0.05), rand(p.D, 8, std=0.05), 8, 16.0)
            p.sync()
        n, ctx = [40, 1, 1, 7], [0, 30, 100, 12]
        self.T = sum(n)
        self.cache = layer.KVCache(40, 16, self.hkv, self.hd)
        self.cache.k.normal_(generator=g)
        self.cache.v.normal_(generator=g)
        self.table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(4, 10)
        self.meta, self.seq = layer.StepMeta(self.T, 1, 8), layer.SeqMeta(4, self.T, 10, self.hq, self.hkv, self.hd)
        self.slots, self.q_start = ints([0] * 30 + [-1] * (self.T - 30)), ints([0, 40, 41, 42, 49])
        self.kv_len = ints([a + b for a, b in zip(n, ctx)])
        self.rope, self.x = layer.Rope(self.hd), rand(self.T, hidden)
        self.build()

    def build(self):
        self.meta.build(self.slots, None, self.pools[0])
        self.seq.build(self.q_start, self.kv_len, self.table, self.T, self.cache, 40)

    def run(self, stream=None):
        return self.layer.attention_block(self.meta, self.seq, self.cache, self.x, self.pools[0], self.W_qkv, self.pools[1],
                                          self.W_o, rope=self.rope, stream=stream)


@pytest.mark.parametrize("raw", [False, True])
def test_attention_block_on_another_stream(layer, raw):
    """The block waits on its stream while the current one makes and fills tensors of its temporaries' sizes; and it runs at
    once while the current stream still has work in memory that was released before the call."""
    b = Block(layer)
    want = b.run()
    sizes = [(b.T * (b.hq + 2 * b.hkv) * b.hd, torch.float32), (b.T * b.hq * b.hd, torch.bfloat16), (b.T * 512, torch.float32)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for late in (True, False):
        if late:
            busy(s)
        else:
            busy(torch.cuda.current_stream())
            for size, dtype in sizes * 3:
                torch.full((size,), float("nan"), dtype=dtype, device="cuda")
        y = b.run(stream=s.cuda_stream if raw else s)
        if late:
            kept = [torch.full((size,), float("nan"), dtype=dtype, device="cuda") for size, dtype in sizes * 3]
        torch.cuda.synchronize()
        assert torch.equal(y, want), late
        del y
    del kept


def test_outputs_made_for_another_stream(layer):
    """Outputs that the calls make while the current stream still has work in memory of their size that was just released."""
    b = Block(layer)
    qkv, rs = torch.randn(b.T, (b.hq + 2 * b.hkv) * b.hd, device="cuda"), ints([0, 40, 71, 172])
    q = layer.qkv_write(b.cache, b.seq, qkv)
    calls = [lambda st: layer.linear(b.pools[0], b.meta, b.x, b.W_qkv, stream=st),
             lambda st: layer.base_gemm(b.x, b.W_qkv, stream=st),
             lambda st: layer.qkv_write(b.cache, b.seq, qkv, stream=st),
             lambda st: layer.attention(b.cache, b.seq, q, stream=st),
             lambda st: layer.kv_read(b.cache, b.seq, rs, 191, stream=st)]
    s = torch.cuda.Stream()
    for call in calls:
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        busy(torch.cuda.current_stream())
        for x in want * 4:
            torch.full_like(x, float("nan"))
        got = call(s)
        torch.cuda.synchronize()
        for x, y in zip(want, got if isinstance(got, tuple) else (got,)):
            assert torch.equal(x, y)


# ------------------------------------------------------------------------------------------- angles
def test_angles_of_fast_frequencies_and_far_positions(layer):
    """Angles of pos * freq radians, freq up to 1e6 and positions up to 2^24, against exact arithmetic: 5e-7 of a radian and a
    few roundings of the fp32 rotation (6e-8 each), in bf16 half a step, 2^-8."""
    from fractions import Fraction
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234136")
    freq = [1e6, 654321.987, 3.0e5, 77777.7, 1234.5678, 31.4, 6.283185, 3.14159, 1.0, 0.7, 0.01, 1e-3, 1e-5, -2.5e5, -1.0, 999999.999]
    rope = layer.Rope(32, freq=freq)
    pos = [0, 1, 2, 3, 1000, 65537, 1 << 20, 16777215, 16777216, 12345678, -5, -16777216]
    T = len(pos)
    st = Step(layer, [T], [0], 1, 1, 128)
    qkv = torch.zeros(T, 3 * 128, device="cuda")
    qkv[:, :16] = 1.0                                     # (1, 0) turned is (cos, sin)
    q = layer.qkv_write(st.cache, st.seq, qkv, rope=rope, positions=ints(pos)).double().cpu().numpy()[:, 0]
    for t, p in enumerate(pos):
        for i, f in enumerate(freq):
            turns = Fraction(p) * Fraction(f) / two_pi
            a = float((turns - round(turns)) * two_pi)
            for got, want in ((q[t, i], np.cos(a)), (q[t, i + 16], np.sin(a))):
                assert abs(got - want) <= 2.0 ** -8 * abs(want) + 1e-6, (p, f, got, want)


# ------------------------------------------------------------------------------------------- refusals
def test_query_and_output_must_not_overlap(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    st = Step(layer, [1, 30], [50, 20])
    both = torch.zeros(2 * st.q.numel(), dtype=torch.bfloat16, device="cuda")
    n = st.q.numel() * 2
    call = lambda q, o: mlora.mlora_attention(st.cache.handle, st.seq.handle, q, 1.0, o)  # noqa: E731
    a = both.data_ptr()
    for q, o in ((a, a), (a, a + 16), (a + n - 16, a), (a, a + n - 16)):
        with pytest.raises(mlora.MloraError) as e:
            call(q, o)
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
    both[:st.q.numel()] = st.q.flatten()
    call(a, a + n)                                        # side by side
    torch.cuda.synchronize()
    assert torch.equal(both[st.q.numel():].view_as(st.run()), st.run(scale=1.0))


def test_outputs_of_the_host_are_refused(layer):
    st = Step(layer, [1, 30], [50, 20])
    host = lambda x: torch.empty(x, dtype=torch.bfloat16)  # noqa: E731
    on = lambda x: host(x).cuda()  # noqa: E731
    with pytest.raises(AssertionError):
        layer.attention(st.cache, st.seq, st.q, host((st.T, st.hq * st.hd)))
    with pytest.raises(AssertionError):
        layer.qkv_write(st.cache, st.seq, torch.zeros(st.T, 12 * 128, device="cuda"), host((st.T, st.hq, st.hd)))
    rows = (sum(st.len), st.hkv, st.hd)
    for k, v in ((host(rows), on(rows)), (on(rows), host(rows))):
        with pytest.raises(AssertionError):
            layer.kv_read(st.cache, st.seq, ints([0, st.len[0]]), rows[0], k, v)


# ------------------------------------------------------------------------------------------- weights
@pytest.mark.parametrize("n,ctx,hq,hkv,hd", [([1] * 5, [700, 64, 3, 2000, 150], 8, 2, 128), ([1, 1], [300, 9000], 4, 1, 64),
                                             ([2, 1, 2], [500, 90, 1200], 8, 2, 128), ([3, 4, 1], [100, 900, 200], 8, 2, 64),
                                             ([1, 1], [700, 40], 16, 1, 128)])
def test_weights_of_few_rows_keep_16_bits(layer, n, ctx, hq, hkv, hd):
    """bf16, sequences of few rows: the weights are two bf16 numbers, the second rounded at 2^-8 of 2^-8 of the first."""
    from oracle import attention as ref
    st = Step(layer, n, ctx, hq, hkv, hd, seed=13)
    o = st.run()
    want, W, S = ref.attention(st.q.double().cpu().numpy(), [r[0] for r in st.rows], [r[1] for r in st.rows], st.starts, hq // hkv, hd ** -0.5)
    got = o.double().cpu().numpy().reshape(want.shape)
    d = (hd * 2.0 ** -24 + 2.0 ** -20) * S[..., None]
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -16 + 2 * d) * (W + np.abs(want)) + 1e-30
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.nanmax(np.abs(got - want) / tol)))


def test_whole_blocks_dealt_out_over_e4m3(layer):
    """200 short chunks, dealt out whole, head size 64, over e4m3 with scores (checked here) that leave every weight above 2^-24 of
    its row's largest, and value scales that differ by at most 2^6: nothing rests on what is below f16's range."""
    from tests.test_gpu_attention import DEALT
    n, ctx, hq, hkv, hd = DEALT[1]
    assert hq == hkv
    st = Step(layer, n, ctx, hq, hkv, hd, 32, "e4m3", seed=21)
    rng = np.random.default_rng(2)
    table = st.table.cpu().numpy()
    for which, (x, z, lo, hi) in enumerate(((st.k, st.ks, -10.0, -7.5), (st.v, st.vs, -8.0, -2.0))):
        z.copy_(torch.where(torch.isnan(z), z, torch.from_numpy(2.0 ** rng.uniform(lo, hi, tuple(z.shape))).to(z)))
        code, scale = x.double().cpu().numpy(), z.double().cpu().numpy()
        for s, L in enumerate(st.len):
            p, off = table[s, np.arange(L) // 32], np.arange(L) % 32
            st.rows[s][which] = code[p, :, off] * scale[p, :, off][..., None]
    q = st.q.double().cpu().numpy()
    for s in range(len(n)):
        z = np.einsum("thd,jhd->thj", q[st.starts[s]:st.starts[s + 1]], st.rows[s][0]) * hd ** -0.5
        assert np.ptp(z, axis=-1).max() < 24 * np.log(2)
    o = st.run()
    st.seq.status()
    st.check(o)
    for _ in range(2):
        st.build()
        assert torch.equal(o, st.run())


@pytest.mark.parametrize("n,ctx,hq,hkv,hd", [([366, 127, 33], [0, 0, 0], 6, 2, 128), ([23, 1, 60], [42, 7, 2904], 7, 1, 64), ([368], [0], 99, 3, 128)])
def test_chunks_of_odd_groups_repeat_their_bits(layer, n, ctx, hq, hkv, hd):
    """Groups that do not divide a tile of 128 rows leave rows of it without a token, in which the shared memory's earlier content
    stays: whatever other calls have left there, a call over e4m3 repeats its bits."""
    st = Step(layer, n, ctx, hq, hkv, hd, kind="e4m3", seed=3, q_gain=0.002)
    o = st.run()
    st.seq.status()
    st.check(o)
    other = Step(layer, [300], [200], 8, 2, hd, kind="e4m3", seed=4, q_gain=300.0)
    for _ in range(6):
        other.run()
        assert torch.equal(o, st.run())
        other.q.neg_()
        assert torch.equal(o, st.run())
