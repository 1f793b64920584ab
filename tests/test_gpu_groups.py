"""Attention of groups of sequences behind a shared prefix, against fp64, element by element. The sums over the prefix and over a
sequence's own keys are those of the plain attention's kernels, joined in fp32, so that its tolerances (test_gpu_attention.py)
hold. Groups are a hint: what is computed never depends on them."""
import numpy as np
import pytest

from tests.test_gpu_attention import Step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

WIDE = 1 << 15          # entries of a page table's row: by them the prefixes might be long enough to be worth a pass


@pytest.fixture(scope="module")
def layer():
    from rank_adapter_gemm_token_gb300 import layer
    return layer


class Groups(Step):
    """groups: (first sequence, one past the last, prefix) of each; their sequences hold the prefix's whole pages in common."""

    def __init__(self, layer, n, ctx, hq=8, hkv=2, hd=128, page=16, kind="bf16", groups=(), apart=(), **kw):
        self.groups = groups
        self.bounds = None
        super().__init__(layer, n, ctx, hq, hkv, hd, page, kind, **kw)
        wide = torch.full((len(n), WIDE), -1, dtype=torch.int32, device="cuda")
        wide[:, :self.table.shape[1]] = self.table
        self.table = wide
        for a, b, prefix in groups:
            for s in range(a + 1, b):
                whole = min(prefix, self.len[s], self.len[a]) // page
                if s in apart or whole == 0:
                    continue
                old = self.table[s, :whole].clone().long()
                self.table[s, :whole] = self.table[a, :whole]
                for x in (self.k, self.v):               # the pages that it gives back are not read
                    x.view(torch.uint8)[old] = 127 if kind == "e4m3" else 255
                for side in (0, 1):
                    self.rows[s][side] = self.rows[s][side].copy()
                    self.rows[s][side][:whole * page] = self.rows[a][side][:whole * page]
        self.seq = layer.SeqMeta(len(n), max(self.T, 1), WIDE, hq, hkv, hd, max_groups=max(len(groups), 1))
        starts = []
        for a, b, _ in groups:
            assert not starts or starts[-1] == a, "groups one after another"
            starts += [a, b] if not starts else [b]
        self.group_start = torch.tensor(starts or [0], dtype=torch.int32, device="cuda")
        self.prefix_len = torch.tensor([p for _, _, p in groups], dtype=torch.int32, device="cuda")
        self.build()

    def build(self, **kw):
        if not hasattr(self, "prefix_len"):
            return super().build()
        self.seq.build(self.q_start, self.kv_len, self.table, self.T, self.cache, self.max_new, group_start=self.group_start,
                       prefix_len=self.prefix_len, **kw)

    def launches(self):
        from rank_adapter_gemm_token_gb300 import mlora
        before = mlora.mlora_launch_count()
        self.run()
        return mlora.mlora_launch_count() - before


CASES = [
    # new, behind the start (prefix among it), heads, kv heads, hd, page, groups
    ([1] * 4, [300, 280, 256, 299], 8, 2, 128, 16, [(0, 4, 256)]),
    ([1] * 4, [300, 280, 256, 299], 8, 2, 64, 8, [(0, 4, 255)]),                        # 128 of them are shared
    ([1] * 9, [700 + 9 * i for i in range(9)], 32, 8, 128, 32, [(0, 3, 600), (3, 9, 650)]),
    ([1] * 7, [520] * 7, 16, 1, 128, 16, [(0, 5, 512)]),                                # two of none
    ([1] * 6, [900, 900, 1000, 901, 902, 40], 7, 1, 128, 64, [(0, 2, 128), (2, 6, 896)]),      # the last is shorter than the prefix
    ([1, 2, 3, 1], [400] * 4, 4, 4, 64, 256, [(0, 4, 400)]),                            # pages longer than a key tile
    ([1, 0, 1, 0, 2], [300, 300, 0, 0, 290], 8, 2, 128, 16, [(0, 5, 288)]),             # no new tokens, a first token, an empty one
    ([40, 1, 70, 33], [512, 512, 530, 512], 8, 2, 128, 16, [(0, 4, 512)]),              # chunks and a token
    ([200, 300, 64], [384, 400, 390], 28, 4, 128, 128, [(0, 3, 384)]),
    ([130] * 3, [256] * 3, 24, 1, 64, 32, [(0, 3, 256)]),
    ([12] * 5, [256] * 5, 24, 1, 64, 32, [(0, 5, 256)]),
    ([1] * 130, [140 + i % 7 for i in range(130)], 8, 2, 128, 16, [(0, 2, 128), (2, 100, 140), (100, 101, 130), (101, 130, 139)]),
    ([1] * 3, [5000, 5100, 4999], 8, 2, 128, 64, [(0, 3, 4992)]),                       # the prefix's keys are split among CTAs
    ([3] * 5, [2000] * 5, 12, 12, 64, 16, [(0, 5, 1990)]),
    ([1] * 5, [100] * 5, 8, 2, 128, 16, [(0, 5, 100)]),                                 # below 128: nothing is shared
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_groups(layer, case, kind):
    n, ctx, hq, hkv, hd, page, groups = CASES[case]
    st = Groups(layer, n, ctx, hq, hkv, hd, page, kind, groups, seed=case, tail=2, lead=1)
    assert st.launches() >= 3                           # the prefixes' pass and its join beside the others
    o = st.run()
    st.seq.status()
    st.check(o)
    assert (o[0] == 0).all() and (o[-2:] == 0).all()
    for _ in range(2):
        st.build()
        assert torch.equal(o, st.run()), "a repeated call differs"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_scores(layer, kind):
    """Scores of tens to hundreds, so that the prefix or the own keys carry nearly all of a row's weight."""
    st = Groups(layer, [1, 1, 50, 1], [400, 420, 390, 600], groups=[(0, 4, 384)], kind=kind, seed=3, q_gain=20.0)
    st.check(st.run())


def test_what_does_not_share_stands_alone(layer):
    """Members with other pages, or whose prefix is not cached yet; a first sequence that is padding, or rejected."""
    from rank_adapter_gemm_token_gb300 import mlora
    n, ctx = [1, 1, 60, 1, 1], [400, 410, 300, 420, 400]
    st = Groups(layer, n, ctx, groups=[(0, 5, 384)], apart=(3,))
    st.check(st.run())
    st.seq.status()
    first = Groups(layer, n, ctx, groups=[(0, 5, 384)])
    want = first.run()
    first.check(want)
    first.kv_len[0] = 0                                 # padding: its pages still say what is shared
    first.build()
    o = first.run()
    first.seq.status()
    assert (o[0] == 0).all()
    first.rows[0] = [r[:0] for r in first.rows[0]]
    first.check(o)
    first.kv_len[0] = -1
    first.build()
    o = first.run()
    with pytest.raises(mlora.MloraError) as e:
        first.seq.status()
    assert e.value.status == mlora.MLORA_ERR_BAD_SEQUENCE
    first.check(o)
    first.table[0, :24] = -7                            # the first one's pages do not hold, nor are they anyone's
    first.build()
    o = first.run()
    with pytest.raises(mlora.MloraError):
        first.seq.status()
    first.check(o)


def test_bounds_that_do_not_ascend(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    st = Groups(layer, [1] * 6, [300] * 6, groups=[(0, 3, 256), (3, 6, 288)])
    st.check(st.run())
    for bad in ([3, 0, 6], [0, 7, 6], [0, 3, 7], [-1, 3, 6], [0, 3, 2 ** 31 - 1]):
        st.group_start.copy_(torch.tensor(bad, dtype=torch.int32))
        st.build()
        st.check(st.run())
        with pytest.raises(mlora.MloraError) as e:
            st.seq.status()
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG and "groups" in str(e.value)
    st.group_start.copy_(torch.tensor([0, 3, 6], dtype=torch.int32))
    for bad in ([-5, 2 ** 31 - 1], [0, -2 ** 31], [10 ** 6, 300]):
        st.prefix_len.copy_(torch.tensor(bad, dtype=torch.int32))
        st.build()
        st.check(st.run())
        st.seq.status()


def test_starts_that_fall_inside_a_group(layer):
    """Starts that fall inside a group: its first sequence alone stands."""
    from rank_adapter_gemm_token_gb300 import mlora
    st = Groups(layer, [5, 1, 8, 1, 4], [300, 310, 299, 300, 305], groups=[(0, 5, 288)])
    st.q_start[2] = 19                                  # sequence 1 gets 13 tokens, above max_new; 2 falls back to 14
    st.build()
    o = st.run()
    with pytest.raises(mlora.MloraError):
        st.seq.status()
    st.starts, st.rows = [0, 5], st.rows[:1]
    st.check(o)


def test_small_savings_take_no_pass(layer):
    st = Groups(layer, [1] * 4, [300] * 4, groups=[(0, 4, 256)])
    with_pass = st.launches()
    o = st.run()
    st.build(max_prefix=256)
    assert st.launches() == with_pass - 2
    st.check(st.run())
    st.check(o)
    st.build(max_prefix=0)
    st.check(st.run())


def test_no_groups_and_plain_builds_between(layer):
    st = Groups(layer, [1, 30, 1], [300, 300, 300], groups=[(0, 3, 288)])
    a = st.run()
    Step.build(st)
    plain = st.run()
    st.check(plain)
    st.seq.build(st.q_start, st.kv_len, st.table, st.T, st.cache, st.max_new, group_start=st.group_start[:1], prefix_len=st.prefix_len[:0])
    assert torch.equal(plain, st.run())
    st.build()
    assert torch.equal(a, st.run())
    st.seq.build(st.q_start, st.kv_len, st.table, st.T, st.cache, st.max_new, window=10 ** 6)
    st.check(st.run())


def test_values_that_are_not_finite(layer):
    """A NaN in a sequence's own keys reaches its rows alone; one in the prefix's reaches the group's."""
    st = Groups(layer, [1] * 6, [300] * 6, groups=[(0, 3, 256), (3, 6, 256)])
    good = st.run()
    st.k[int(st.table[1, 290 // 16]), :, 290 % 16] = float("nan")
    o = st.run()
    assert o[1].isnan().all() and torch.equal(o[[0, 2, 3, 4, 5]], good[[0, 2, 3, 4, 5]])
    st.v[int(st.table[3, 3]), :, 5] = float("nan")
    o = st.run()
    assert o[[1, 3, 4, 5]].isnan().all() and torch.equal(o[[0, 2]], good[[0, 2]])


def test_graph_replay_and_streams(layer):
    steps = [Groups(layer, [1, 30, 2, 1], [400, 400, 390, 401], groups=[(0, 2, 384), (2, 4, 380)], seed=s) for s in (1, 2)]
    out = [torch.empty(st.T, st.hq * st.hd, dtype=torch.bfloat16, device="cuda") for st in steps]
    graphs, s = [], torch.cuda.Stream()
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
    steps[0].prefix_len[0] = 256                        # the arrays are read at each replay
    steps[0].group_start[1] = 0
    graphs[0].replay()
    torch.cuda.synchronize()
    steps[0].check(out[0])
    st, want = steps[1], steps[1].run()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    st.build(stream=other)
    got = layer.attention(st.cache, st.seq, st.q, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(got, want)


def test_refusals(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    st = Groups(layer, [1] * 4, [300] * 4, groups=[(0, 4, 256)])
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def refused(status, *, groups=st.group_start, prefixes=st.prefix_len, count=1, most=1000):
        with pytest.raises(mlora.MloraError) as e:
            mlora.mlora_build_seq_groups(st.seq.handle, st.q_start, st.kv_len, st.table, WIDE, 4, 4, 1, groups, prefixes, count, most,
                                         st.cache.handle)
        assert e.value.status == status

    refused(mlora.MLORA_ERR_INVALID_ARG, groups=None)
    refused(mlora.MLORA_ERR_INVALID_ARG, prefixes=None)
    refused(mlora.MLORA_ERR_INVALID_ARG, count=-1)
    refused(mlora.MLORA_ERR_INVALID_ARG, most=-1)
    refused(mlora.MLORA_ERR_TOO_MANY_TOKENS, groups=ints([0, 1, 4]), prefixes=ints([256, 256]), count=2)
    with pytest.raises(mlora.MloraError):
        layer.SeqMeta(4, 4, 100, 8, 2, 128, max_groups=5)
    with pytest.raises(mlora.MloraError):
        layer.SeqMeta(4, 4, 100, 8, 2, 128, max_groups=-1)
    for bad in (dict(window=5), dict(sinks=1), dict(prefix_len=st.prefix_len.long()), dict(prefix_len=None),
                dict(group_start=st.group_start.cpu()), dict(group_start=ints([0, 1, 4]))):
        with pytest.raises(AssertionError):
            st.seq.build(st.q_start, st.kv_len, st.table, st.T, st.cache, 1, **{**dict(group_start=st.group_start, prefix_len=st.prefix_len), **bad})
    st.check(st.run())
