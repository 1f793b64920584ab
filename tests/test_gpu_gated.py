"""The gated linear h = act(g) * u over the adapted gate_up projection, against fp64, element by element.

Tolerance, from the arithmetic (a rounding to bf16 is off by at most 2^-8 relative):
  g and u   sums of K exact products in fp32. The tensor cores add 16 products to a sum at a time and may be off by two units
            of 2^-23 of the largest partial sum: (K / 16 + 4) 2^-22 S with S = sum |x_i w_i|, which also covers sums split over
            K. The side path v = A x likewise, over K, and then B v; the scaled v is rounded to bf16: 2^-8 sum_q |B_q v_q|.
  act       its slope is at most 1.13 for the three of them, and |act(g)| <= |g|, so that an error d of g gives 1.13 d; fp32
            with the fast exponential, whose argument up to 90 is off by 2^-23 relative: 2^-14 relative.
  h         the product of both, rounded to bf16: 2^-8 |h|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ACTS = ("silu", "gelu_tanh", "gelu")


@pytest.fixture(scope="module")
def layer():
    from rank_adapter_gemm_token_gb300 import layer
    return layer


def act64(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu_tanh":
        return g / (1 + torch.exp(-2 * (2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    return 0.5 * g * torch.special.erfc(-g * 0.5 ** 0.5)


class Case:
    def __init__(self, layer, T, K, F, slots=4, rank=16, J=1, classes=None, seed=0, gain=1.0, absent=0.2, empty=(), max_tokens=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.layer, self.T, self.K, self.F = layer, T, K, F
        self.x, self.W = rand(T, K, std=gain), rand(2 * F, K, std=K ** -0.5)
        self.pool = layer.AdapterPool(slots, rank, K, 2 * F, classes=classes)
        limit = [r for n, r in classes for _ in range(n)] if classes else [rank] * slots
        n = len(limit)
        self.A, self.B, self.c = [], [], []
        for i, r in enumerate(limit):
            r = max(1, r - i % 3)
            self.A.append(rand(r, K, std=K ** -0.5))
            self.B.append(rand(2 * F, r, std=0.3))
            self.pool.load(i, self.A[i], self.B[i], r, 2.0 * r, rslora=i % 2 == 1)
            self.c.append(2.0 * r / (r ** 0.5 if i % 2 == 1 else r))
        self.pool.sync()
        self.slots = torch.randint(0, n, (T, J), generator=g, device="cuda", dtype=torch.int32)
        self.slots[torch.rand(T, J, generator=g, device="cuda") < absent] = -1
        self.scales = 0.2 + torch.rand(T, J, generator=g, device="cuda")
        self.meta = layer.StepMeta(max_tokens or max(T, 1), J, self.pool.r_max)
        self.build()

    def build(self):
        self.meta.build(self.slots, self.scales, self.pool)

    def run(self, act="silu", **kw):
        h = torch.full((self.T, self.F), 7.0, dtype=torch.bfloat16, device="cuda")
        return self.layer.gated_linear(self.pool, self.meta, self.x, self.W, act=act, h=h, **kw)

    def exact(self):
        """[g u] and the bound of its error."""
        x, W = self.x.double(), self.W.double()
        steps = (self.K / 16 + 4) * 2.0 ** -22
        y, tol = x @ W.T, steps * (x.abs() @ W.abs().T)
        for i, (A, B) in enumerate(zip(self.A, self.B)):
            s = (self.scales.double() * (self.slots == i)).sum(1)[:, None] * self.c[i]
            v, size = s * (x @ A.double().T), s * (x.abs() @ A.double().abs().T)
            y += v @ B.double().T
            tol += (2.0 ** -8 * v.abs() + 2 * steps * size) @ B.double().abs().T * 1.01
        return y, tol

    def check(self, h, act="silu"):
        y, tol = self.exact()
        g, u = y.split(self.F, 1)
        dg, du = tol.split(self.F, 1)
        a = act64(g, act)
        want = a * u
        bound = (1.13 * dg + 2.0 ** -14 * a.abs()) * (u.abs() + du) + a.abs() * du
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 1e-30
        bad = ~((h.double() - want).abs() <= bound)
        assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float(((h.double() - want).abs() / bound).nan_to_num(9e9).max()))


SIZES = [
    # T, K, F, slots, rank, J
    (1, 64, 8, 2, 8, 1),
    (1, 1024, 1000, 4, 16, 1),
    (3, 200, 64, 4, 16, 2),
    (31, 72, 104, 3, 8, 1),
    (64, 512, 4096, 40, 16, 1),
    (127, 256, 96, 8, 64, 1),
    (128, 256, 128, 8, 40, 3),
    (129, 264, 136, 5, 16, 1),
    (255, 64, 512, 100, 8, 1),
    (256, 1024, 2000, 100, 16, 1),
    (257, 320, 200, 7, 16, 8),
    (300, 8, 328, 3, 8, 1),
    (513, 512, 1096, 60, 64, 1),
    (1000, 2048, 24, 9, 64, 2),
    (130, 8200, 72, 4, 16, 1),                       # a K that the pair kernel does not shrink by itself
    (20, 8200, 256, 4, 16, 1),
    (2, 4096, 14336, 4, 16, 1),
    (700, 256, 7000, 16, 32, 1),
]


@pytest.mark.parametrize("case", range(len(SIZES)))
def test_gated_linear(layer, case):
    T, K, F, slots, rank, J = SIZES[case]
    c = Case(layer, T, K, F, slots, rank, J, seed=case)
    act = ACTS[case % 3]
    h = c.run(act)
    c.meta.status()
    c.check(h, act)
    assert torch.equal(h, c.run(act)), "a repeated call differs"


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gain", [1e-3, 1.0, 40.0])
def test_activations(layer, act, gain):
    """Gates near 0, ordinary ones, and those for which the activation has saturated."""
    c = Case(layer, 150, 128, 256, seed=31, gain=gain)
    c.check(c.run(act), act)


@pytest.mark.parametrize("T", [5, 128, 200, 600])
def test_rank_classes(layer, T):
    c = Case(layer, T, 256, 320, classes=[(9, 8), (5, 16), (3, 64), (2, 256)], J=2, seed=T)
    c.check(c.run())
    c.meta.status()


def test_tokens_without_adapters(layer):
    """A step of tokens without adapters, and one token that has one among them."""
    c = Case(layer, 140, 192, 264, absent=2.0, seed=3)
    alone = c.run()
    c.check(alone)
    c.slots[77] = 1
    c.build()
    h = c.run()
    c.check(h)
    keep = torch.arange(140, device="cuda") != 77
    assert torch.equal(h[keep], alone[keep])


def test_more_adapter_blocks_than_a_tile_takes(layer):
    """128 tokens that name 100 adapters of rank 256: 400 column blocks, where the tensor-core side path takes 256."""
    from rank_adapter_gemm_token_gb300 import mlora
    for T in (128, 300):
        c = Case(layer, T, 64, 136, slots=100, rank=256, absent=0.0, seed=T)
        assert mlora.mlora_gated_workspace_bytes(c.pool.handle, c.meta.handle) == T * 272 * 4
        c.check(c.run())
        c.meta.status()


def test_forced_tiles_and_paths(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    c = Case(layer, 200, 256, 328, slots=12, seed=8)
    one = Case(layer, 70, 256, 328, slots=12, seed=9)
    try:
        for n in (-1, 128, 192, 224, 256):
            mlora.mlora_set_gemm_tile_n(n)
            c.check(c.run())
            one.check(one.run())
        mlora.mlora_set_gemm_tile_n(0)
        for path in (1, 2):
            mlora.mlora_set_path(path)
            c.check(c.run())
            one.check(one.run())
    finally:
        mlora.mlora_set_gemm_tile_n(0)
        mlora.mlora_set_path(0)


def test_sliced_adapters(layer):
    """An adapter for each of the two projections, loaded as slices of the stacked linear."""
    from rank_adapter_gemm_token_gb300 import mlora
    T, K, F, r = 90, 128, 160, 8
    c = Case(layer, T, K, F, slots=2, rank=16, seed=4)
    g = torch.Generator().manual_seed(1)
    A = [(torch.randn(r, K, generator=g) * K ** -0.5).to(torch.bfloat16) for _ in range(2)]
    B = [(torch.randn(F, r, generator=g) * 0.3).to(torch.bfloat16) for _ in range(2)]
    mlora.mlora_load_adapter_sliced(c.pool.handle, 0, A, B, r, 2.0 * r, False)
    c.pool.sync()
    c.build()
    c.A[0] = torch.cat(A).cuda()
    whole = torch.zeros(2 * F, 2 * r, dtype=torch.bfloat16)
    whole[:F, :r], whole[F:, r:] = B
    c.B[0], c.c[0] = whole.cuda(), 2.0
    c.check(c.run())


def test_values_that_are_not_finite_stay_in_their_row(layer):
    for T in (40, 180):
        c = Case(layer, T, 128, 136, seed=12)
        good = c.run()
        c.x[7, 5], c.x[20, 9] = float("nan"), float("inf")
        h = c.run()
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[[7, 20]] = False
        assert torch.equal(h[keep], good[keep])
        assert h[7].isnan().all() and not h[20].isfinite().all()


def test_empty_step(layer):
    c = Case(layer, 0, 64, 64, max_tokens=4)
    assert c.run().shape == (0, 64)


def test_rows_behind_and_before_are_left(layer):
    """The output's neighbours in memory: rows past the last token's are not written."""
    for T, F in ((5, 40), (130, 104)):
        c = Case(layer, T, 128, F, seed=2)
        wide = torch.full((T + 400, F), 3.0, dtype=torch.bfloat16, device="cuda")
        layer.gated_linear(c.pool, c.meta, c.x, c.W, h=wide[200:200 + T])
        c.check(wide[200:200 + T])
        assert (wide[:200] == 3).all() and (wide[200 + T:] == 3).all()


def test_another_stream(layer):
    c = Case(layer, 64, 512, 512, seed=6)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = layer.gated_linear(c.pool, c.meta, c.x, c.W, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(h, want)


@pytest.mark.parametrize("T", [16, 300])
def test_graph_replay_follows_the_arrays(layer, T):
    """Two captured steps with the metadata built in them; replayed on other inputs, in either order."""
    cases = [Case(layer, T, 256, 264, seed=s) for s in (1, 2)]
    out = [torch.empty(T, 264, dtype=torch.bfloat16, device="cuda") for _ in cases]
    graphs = []
    stream = torch.cuda.Stream()
    for c, h in zip(cases, out):
        def step():
            c.build()
            layer.gated_linear(c.pool, c.meta, c.x, c.W, h=h)

        with torch.cuda.stream(stream):
            step()                                    # the pool's first use on the stream, outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        graphs.append(graph)
    for k in range(2):
        for c in cases:
            c.x.copy_(torch.randn_like(c.x.float()).to(torch.bfloat16))
            c.slots.copy_(torch.randint_like(c.slots, -1, 4))
        for i in (1, 0, 0, 1):
            graphs[i].replay()
        for c, h in zip(cases, out):
            c.check(h)
            c.meta.status()


def test_feed_forward(layer):
    """Both linears with the activation between them, for decode tokens and a larger batch, on the current stream and another."""
    for T in (9, 260):
        c = Case(layer, T, 256, 512, slots=6, seed=T)
        down = Case(layer, T, 512, 128, slots=6, seed=T + 1)      # (its pool alone: 512 -> 256)
        y = layer.feed_forward(c.meta, c.x, c.pool, c.W, down.pool, down.W)
        g, u = c.exact()[0].split(512, 1)
        down.x, down.slots, down.scales = (act64(g, "silu") * u).to(torch.bfloat16), c.slots, c.scales
        want = down.exact()[0]
        # h is off by a rounding (and where it falls on the other side, by another): 2^-7 of each term at most
        assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -7
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        again = layer.feed_forward(c.meta, c.x, c.pool, c.W, down.pool, down.W, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(again, y)
        c.meta.status()


def test_refusals(layer):
    from rank_adapter_gemm_token_gb300 import mlora
    c = Case(layer, 20, 64, 64, seed=1)
    p, m, h = c.pool.handle, c.meta.handle, torch.empty(20, 64, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(20 * 128 * 4 + 16, dtype=torch.uint8, device="cuda")

    def refused(status, *a):
        with pytest.raises(mlora.MloraError) as e:
            mlora.mlora_gated_linear(*a)
        assert e.value.status == status

    bad = mlora.MLORA_ERR_INVALID_ARG
    refused(bad, 0, m, c.x, c.W, 0, h, work)
    refused(bad, p, 0, c.x, c.W, 0, h, work)
    refused(bad, p, m, None, c.W, 0, h, work)
    refused(bad, p, m, c.x, None, 0, h, work)
    refused(bad, p, m, c.x, c.W, 0, None, work)
    refused(bad, p, m, c.x, c.W, -1, h, work)
    refused(bad, p, m, c.x, c.W, 3, h, work)
    refused(bad, p, m, c.x.data_ptr() + 2, c.W, 0, h, work)
    refused(bad, p, m, c.x, c.W, 0, h.data_ptr() + 8, work)
    refused(bad, p, m, c.x, c.W, 0, c.x, work)
    refused(bad, p, m, c.x, c.W, 0, c.W.data_ptr() + 16, work)
    odd = layer.AdapterPool(4, 16, 64, 136)            # half of 136 is no multiple of 8
    refused(bad, odd.handle, m, c.x, c.W, 0, h, work)
    other = layer.AdapterPool(5, 16, 64, 128)
    refused(mlora.MLORA_ERR_MISMATCH, other.handle, m, c.x, c.W, 0, h, work)
    table = layer.EmbeddingPool(64, 128, [(4, 16)])
    refused(bad, table.handle, m, c.x, c.W, 0, h, work)
    fresh = layer.StepMeta(4, 1, 16)
    refused(bad, p, fresh.handle, c.x, c.W, 0, h, work)
    with pytest.raises(KeyError):
        layer.gated_linear(c.pool, c.meta, c.x, c.W, act="tanh")
    with pytest.raises(AssertionError):
        layer.gated_linear(c.pool, c.meta, c.x.float(), c.W)
    with pytest.raises(AssertionError):
        layer.gated_linear(c.pool, c.meta, c.x, c.W, h=torch.empty(20, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(AssertionError):
        layer.gated_linear(c.pool, c.meta, c.x.cpu(), c.W)
    over = layer.AdapterPool(100, 256, 64, 272)        # a step that needs the workspace
    for i in range(100):
        over.load(i, torch.zeros(256, 64, dtype=torch.bfloat16), torch.zeros(272, 256, dtype=torch.bfloat16), 256, 1.0)
    over.sync()
    meta = layer.StepMeta(128, 1, 256)
    meta.build(torch.arange(128, dtype=torch.int32, device="cuda") % 100, None, over)
    x, W, h = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in (128 * 64, 272 * 64, 128 * 136))
    refused(bad, over.handle, meta.handle, x, W, 0, h, None)


FEW = [(T, J) for T in (1, 2, 8, 9, 16, 17, 31, 32, 33, 64) for J in (1, 3)] + [(5, 8), (32, 8)]


@pytest.mark.parametrize("T,J", FEW)
def test_few_tokens(layer, T, J):
    """The kernel of a few tokens: from one share of the side path to more than there are CTAs, slots named twice by a token, K
    that ends inside a step, one group of columns and many."""
    for K, F, slots, rank in ((8, 8, 1, 8), (1000, 72, 5, 40), (264, 9000, 40, 16), (64, 136, 300, 64)):
        c = Case(layer, T, K, F, slots, rank, J, seed=T + J)
        h = c.run("gelu")
        c.meta.status()
        c.check(h, "gelu")
        assert torch.equal(h, c.run("gelu")), "a repeated call differs"


def test_few_tokens_between_other_kernels_on_their_metadata(layer):
    """The linear's tensor-core path and the few tokens' kernel count in the same places: each leaves them as it found them."""
    c = Case(layer, 20, 256, 512, classes=[(9, 8), (5, 16), (3, 64)], J=2, seed=5)
    down = Case(layer, 20, 512, 128, classes=[(9, 8), (5, 16), (3, 64)], J=2, seed=6)
    first = c.run()
    c.check(first)
    for _ in range(3):
        y = layer.feed_forward(c.meta, c.x, c.pool, c.W, down.pool, down.W)
        assert torch.equal(c.run(), first)
        assert torch.equal(y, layer.feed_forward(c.meta, c.x, c.pool, c.W, down.pool, down.W))
    c.meta.status()


def test_slots_cleared_behind_the_metadata(layer):
    """Slots that were loaded when the metadata was built and are empty when the linear runs add nothing, and nothing waits."""
    for T in (1, 12, 200):
        c = Case(layer, T, 128, 264, slots=6, seed=T)
        for s in range(6):
            c.pool.clear(s)
        c.pool.sync()
        for _ in range(2):
            h = c.run()
        c.meta.status()
        c.A, c.B = [a * 0 for a in c.A], [b * 0 for b in c.B]
        c.check(h)


def test_two_streams_at_once(layer):
    """Steps with metadata and pools of their own, side by side on two streams: CTAs of both share the GPU."""
    cases = [Case(layer, T, 2048, 4096, slots=30, rank=64, seed=T) for T in (30, 31)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(cases, streams)):
            got[i].append(layer.gated_linear(c.pool, c.meta, c.x, c.W, stream=s))
    torch.cuda.synchronize()
    for i, c in enumerate(cases):
        c.check(want[i])
        assert all(torch.equal(h, want[i]) for h in got[i])
        c.meta.status()
