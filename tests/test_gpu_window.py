"""Attention over a window and a few first tokens, against fp64, element by element: the tolerances of the plain attention
(test_gpu_attention.py). Whatever no token of a step sees is NaN, or on pages that are gone."""
import numpy as np
import pytest

from oracle import attention as ref
from tests.test_gpu_attention import CASES, Step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layer():
    from rank_adapter_gemm_token_gb300 import layer
    return layer


class Window(Step):
    def __init__(self, layer, n, ctx, hq=8, hkv=2, hd=128, page=16, kind="bf16", window=100, sinks=4, spoil=True, **kw):
        self.window, self.sinks = window, sinks
        super().__init__(layer, n, ctx, hq, hkv, hd, page, kind, **kw)
        if spoil:
            self.spoil()
            self.build()

    def hidden(self, s):
        """Positions of sequence s that none of its new tokens sees."""
        first = max(0, self.len[s] - self.n[s] - self.window + 1)
        return np.arange(min(self.sinks, first), first)

    def spoil(self):
        gone = (-1, 2 ** 30, -2 ** 31)
        self.held = []
        for s in range(len(self.n)):
            rows = self.hidden(s)
            table, off = self.table[s].cpu().numpy()[rows // self.page], rows % self.page
            for x, z in ((self.k, self.ks), (self.v, self.vs)):
                if self.kind == "e4m3":
                    x.view(torch.uint8)[table, :, off] = 127
                    z[table, :, off] = float("nan")
                else:
                    x[table, :, off] = float("nan")
            pages, counts = np.unique(rows // self.page, return_counts=True)
            pages = pages[counts == self.page]
            self.held.append(np.setdiff1d(np.arange(self.len[s]), (pages[:, None] * self.page + np.arange(self.page)).ravel()))
            for i, p in enumerate(pages):
                self.table[s, p] = gone[i % 3]

    def build(self):
        self.seq.build(self.q_start, self.kv_len, self.table, self.T, self.cache, self.max_new, window=self.window, sinks=self.sinks)

    def check(self, o, scale=None):
        scale = self.hd ** -0.5 if scale is None else scale
        want, W, S = ref.attention(self.q.double().cpu().numpy(), [r[0] for r in self.rows], [r[1] for r in self.rows],
                                   self.starts, self.hq // self.hkv, scale, self.window, self.sinks)
        got = o.double().cpu().numpy().reshape(want.shape)
        up, uq = (2.0 ** -8, 0.0) if self.kind == "bf16" else (2.0 ** -11, 2.0 ** -11)
        d = (uq + self.hd * 2.0 ** -24 + 2.0 ** -20) * S[..., None]
        tol = 2.0 ** -8 * np.abs(want) + (up + 2 * d) * (W + np.abs(want)) + 1e-30
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(got - want) / tol)))


WINDOWS = [(1, 0), (1, 1), (5, 4), (16, 0), (64, 64), (100, 4), (128, 0), (129, 130), (500, 70), (1 << 30, 9)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_window(layer, case, kind):
    n, ctx, hq, hkv, hd, page = CASES[case]
    for i in range(3):
        window, sinks = WINDOWS[(3 * case + i) % len(WINDOWS)]
        st = Window(layer, n, ctx, hq, hkv, hd, page, kind, window, sinks, seed=case)
        o = st.run()
        st.seq.status()
        st.check(o)
        assert torch.equal(o, st.run()), "a repeated call differs"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(40, 0), (40, 4), (64, 64), (65, 63), (100, 65), (128, 128), (200, 130), (300, 1), (1000, 20)])
def test_chunks_and_tokens_far_into_a_sequence(layer, window, sinks, kind):
    """Single tokens, few tokens and chunks on contexts around the window's length and far beyond, pages from 8 to 256."""
    for page, hq, hkv, hd in ((8, 8, 2, 128), (64, 4, 4, 64), (256, 16, 1, 128)):
        st = Window(layer, [1, 1, 2, 150, 1, 70, 300], [window - 1, 1500, window + 63, 700, sinks + window, 0, 77], hq, hkv, hd, page, kind,
                    window, sinks, seed=window + sinks, tail=3, lead=2)
        o = st.run()
        st.seq.status()
        st.check(o)
        assert (o[:2] == 0).all() and (o[-3:] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n,ctx,hq,hkv,window,sinks", [([1], [20000], 4, 1, 9000, 200), ([3], [7000], 4, 1, 6001, 4), ([9], [6000], 4, 1, 3500, 0),
                                                       ([70], [4000], 4, 2, 2500, 130), ([5, 1, 1], [3100, 8000, 1], 8, 1, 2000, 70)])
def test_long_windows_are_split_and_joined(layer, n, ctx, hq, hkv, window, sinks, kind):
    st = Window(layer, n, ctx, hq, hkv, kind=kind, page=64, window=window, sinks=sinks, seed=5)
    o = st.run()
    st.seq.status()
    st.check(o)
    for _ in range(3):
        assert torch.equal(o, st.run()), "the parts' order changes the result"


def test_whole_blocks_dealt_out(layer):
    st = Window(layer, [700, 90, 333, 512, 61, 900, 40], [0, 300, 0, 64, 700, 0, 129], 32, 8, 128, 32, window=190, sinks=33, seed=2)
    o = st.run()
    st.seq.status()
    st.check(o)
    for _ in range(3):
        st.build()
        assert torch.equal(o, st.run()), "who takes a block changes the result"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_one_object_for_windows_and_whole_contexts(layer, kind):
    """Builds of either kind after one another on one object, over a cache that holds everything."""
    st = Window(layer, [1, 60, 2], [500, 300, 90], kind=kind, window=77, sinks=3, spoil=False)
    near = st.run()
    st.check(near)
    Step.build(st)
    far = st.run()
    Step.check(st, far)
    st.build()
    assert torch.equal(near, st.run())
    st.window = 10 ** 6
    st.build()
    st.check(st.run())


def test_read_leaves_pages_that_are_gone(layer):
    for kind in ("bf16", "e4m3"):
        st = Window(layer, [1, 0, 40], [300, 95, 200], page=16, kind=kind, window=50, sinks=20)
        start = [3]
        for x in st.len:
            start.append(start[-1] + x + 2)
        rows = start[-1] + 4
        k, v = (torch.full((rows, st.hkv, st.hd), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        layer.kv_read(st.cache, st.seq, torch.tensor(start, dtype=torch.int32, device="cuda"), rows, k, v)
        st.seq.status()
        left = np.ones(rows, bool)
        for s in range(3):
            at, sure = start[s] + st.held[s], ~np.isin(st.held[s], st.hidden(s))
            left[at] = False
            for got, want in ((k, st.rows[s][0]), (v, st.rows[s][1])):
                want = torch.from_numpy(want[st.held[s][sure]]).to(torch.bfloat16)
                assert torch.equal(got[torch.from_numpy(at[sure]).cuda()].cpu(), want)
        assert (k[torch.from_numpy(left).cuda()] == 5).all() and (v[torch.from_numpy(left).cuda()] == 5).all()


def test_written_token_by_token(layer):
    """A sequence written and attended a chunk at a time over a ring of pages: pages that the window has left are given to the
    positions ahead. The last tokens' rows are those of the sequence in one step."""
    hq, hkv, hd, page, window, sinks = 8, 2, 64, 16, 50, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    n = [30, 1, 1, 40, 17, 1, 60, 1, 9, 33]
    L = sum(n)
    qkv = torch.randn(L, (hq + 2 * hkv) * hd, generator=g, device="cuda")
    rope = layer.Rope(hd)
    pages = -(-L // page)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(cache, seq, rows, length, table):
        seq.build(ints([0, len(rows)]), ints([length]), table, len(rows), cache, max_new=len(rows), window=window, sinks=sinks)
        o = layer.attention(cache, seq, layer.qkv_write(cache, seq, rows, rope=rope))
        seq.status()
        return o

    whole = layer.KVCache(pages, page, hkv, hd)
    want = step(whole, layer.SeqMeta(1, L, pages, hq, hkv, hd), qkv, L, ints([list(range(pages))]))
    ring = 1 + (window + max(n)) // page + 2
    cache, seq = layer.KVCache(ring, page, hkv, hd), layer.SeqMeta(1, L, pages, hq, hkv, hd)
    got, at = [], 0
    for k in n:
        table = [-1] * pages
        for i in range(-(-(at + k) // page)):
            if i * page < sinks:
                table[i] = i
            elif (i + 1) * page > at - window + 1:
                table[i] = 1 + (i - 1) % (ring - 1)
        got.append(step(cache, seq, qkv[at:at + k], at + k, ints([table])))
        at += k
    a, b = torch.cat(got).double(), want.double()
    # both are within a few roundings of 2^-8 of the exact rows; their weights' roundings differ by kernel
    assert float((a - b).norm() / b.norm()) < 2.0 ** -7


def test_offsets_past_32_bits(layer):
    """Pages more than 2^32 bytes into the cache."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("memory")
    st = Window(layer, [1, 40], [400, 300], hkv=8, hq=8, page=256, n_pages=9000, window=90, sinks=5)
    st.check(st.run())


def test_graph_replay_and_streams(layer):
    """Two captured steps with one workspace each, replayed out of order on changed tables; and a step on another stream."""
    steps = [Window(layer, [1, 30, 2], [200, 40, 600], window=w, sinks=5, seed=w, spoil=False) for w in (48, 100)]
    out = [torch.empty(st.T, st.hq * st.hd, dtype=torch.bfloat16, device="cuda") for st in steps]
    graphs = []
    s = torch.cuda.Stream()
    for st, o in zip(steps, out):
        run = lambda: (st.build(), layer.attention(st.cache, st.seq, st.q, o))  # noqa: E731
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run()
        graphs.append(g)
    for i in (1, 0, 1, 0):
        out[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        steps[i].check(out[i])
    st = steps[0]
    st.kv_len[0] = 120                                  # the cache holds more of this one than the step now has
    st.len[0], st.rows[0] = 120, [r[:120] for r in st.rows[0]]
    graphs[0].replay()
    torch.cuda.synchronize()
    st.check(out[0])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    st = steps[1]
    want = st.run()
    st.seq.build(st.q_start, st.kv_len, st.table, st.T, st.cache, st.max_new, stream=other, window=st.window, sinks=st.sinks)
    got = layer.attention(st.cache, st.seq, st.q, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got, want)


def test_rejected_sequences(layer):
    """A page outside the cache counts where it is seen alone; the others of the step stand."""
    from rank_adapter_gemm_token_gb300 import mlora
    st = Window(layer, [1, 1, 1], [300, 300, 300], page=16, window=40, sinks=4)
    want = st.run()
    st.table[1, 300 // 16] = 10 ** 6
    st.build()
    o = st.run()
    with pytest.raises(mlora.MloraError) as e:
        st.seq.status()
    assert e.value.status == mlora.MLORA_ERR_BAD_SEQUENCE and "sequence 1" in str(e.value)
    assert (o[1] == 0).all() and torch.equal(o[0], want[0]) and torch.equal(o[2], want[2])


def test_refusals(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    st = Window(layer, [1], [30])
    for window, sinks in ((0, 0), (-3, 0), (5, -1), (5, mlora.MLORA_MAX_SINKS + 1)):
        with pytest.raises(mlora.MloraError) as e:
            st.seq.build(st.q_start, st.kv_len, st.table, st.T, st.cache, 1, window=window, sinks=sinks)
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
    with pytest.raises(AssertionError):
        st.seq.build(st.q_start, st.kv_len, st.table, st.T, st.cache, 1, sinks=4)
    with pytest.raises(mlora.MloraError):
        mlora.mlora_build_seq_window(0, st.q_start, st.kv_len, st.table, st.table.shape[1], 1, 1, 1, 5, 0, st.cache.handle)
    st.check(st.run())                                  # what was built before still stands
