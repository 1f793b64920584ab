"""A local layer (window, first tokens) and a global one, each an attention block and a feed-forward block with adapters, serving
sequences behind a shared prefix: the prefix in one step, the sequences' own prompts in the next, then single tokens. Every
token's output is compared with fp64 over its whole sequence, with bf16 roundings where the operators pass bf16 on.

Tolerance: what the operators pass on is rounded to bf16 (q, k, v, the attention's output, h, x), 2^-8 of each value at most, and
the attention's weights too. How far that carries depends on the step: the adapters here are as large as the base weights, and the
second layer's scores reach a hundred, where a rounded q or k moves a weight by a third. So the same fp64 model is run again
eight times with every rounding replaced by one that is off by a random part of 2^-8 (of e4m3 keys and values: 2^-4), and a row
may differ by four times the most that any of these runs differ in it, plus 2^-6 of its norm.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HIDDEN, HQ, HKV, HD, F, PAGE = 256, 8, 2, 64, 512, 16
QKV, RANK, SLOTS = (HQ + 2 * HKV) * HD, 8, 4
WINDOW, SINKS, PREFIX = 48, 5, 264
OWN, NEW = (9, 1, 30, 17, 70, 4), 3


@pytest.fixture(scope="module")
def layer():
    from rank_adapter_gemm_token_gb300 import layer
    return layer


class Linear:
    def __init__(self, layer, rand, K, D):
        self.W = rand(D, K, std=K ** -0.5)
        self.A, self.B = [rand(RANK, K, std=K ** -0.5) for _ in range(SLOTS)], [rand(D, RANK, std=0.2) for _ in range(SLOTS)]
        self.pool = layer.AdapterPool(SLOTS, RANK, K, D)
        for s in range(SLOTS):
            self.pool.load(s, self.A[s], self.B[s], RANK, 2.0 * RANK)
        self.pool.sync()

    def exact(self, x, slot):
        y = x @ self.W.double().T
        return y if slot < 0 else y + 2.0 * (x @ self.A[slot].double().T) @ self.B[slot].double().T


def exact_block(x, slot, lin, window, rope, bf, kv):
    """One layer over a whole sequence: x [L, HIDDEN] in 64 bits, the attention block and the feed-forward block with a residual
    around each; bf rounds what is passed on, kv what goes to the cache."""
    L = len(x)
    q, k, v = lin["qkv"].exact(x, slot).view(L, HQ + 2 * HKV, HD).split((HQ, HKV, HKV), 1)
    ang = torch.arange(L, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(rope.freq, device="cuda", dtype=torch.float64)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

    def turn(y):
        a, b = y.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    q, k, v = bf(turn(q)), kv(turn(k)), kv(v)
    k, v = (t.repeat_interleave(HQ // HKV, 1) for t in (k, v))
    z = torch.einsum("thd,khd->htk", q, k) / math.sqrt(HD)
    p, j = torch.arange(L, device="cuda")[:, None], torch.arange(L, device="cuda")[None]
    hide = j > p
    if window:
        hide |= (j >= SINKS) & (j <= p - WINDOW)
    o = torch.einsum("htk,khd->thd", torch.softmax(z.masked_fill(hide, -math.inf), -1), v).reshape(L, -1)
    x = bf(x + lin["o"].exact(bf(o), slot))
    g, u = lin["up"].exact(x, slot).split(F, 1)
    return bf(x + lin["down"].exact(bf(g * torch.sigmoid(g) * u), slot))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_served_together(layer, kind):
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    lins = [{"qkv": Linear(layer, rand, HIDDEN, QKV), "o": Linear(layer, rand, HQ * HD, HIDDEN),
             "up": Linear(layer, rand, HIDDEN, 2 * F), "down": Linear(layer, rand, F, HIDDEN)} for _ in range(2)]
    rope = layer.Rope(HD)
    n = len(OWN)
    slot_of = [-1] + [i % SLOTS for i in range(n - 1)]
    common = rand(PREFIX, HIDDEN)
    own = [rand(k + NEW, HIDDEN) for k in OWN]
    lens = [PREFIX + k + NEW for k in OWN]
    whole = PREFIX // PAGE
    most = -(-max(lens) // PAGE)
    n_pages = whole + sum(-(-L // PAGE) - whole for L in lens)
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    caches = [layer.KVCache(n_pages, PAGE, HKV, HD, dtype) for _ in range(2)]
    free = list(range(n_pages))[::-1]
    shared = [free.pop() for _ in range(whole)]
    table = []
    for L in lens:
        table.append(shared + [free.pop() for _ in range(-(-L // PAGE) - whole)])
        table[-1] += [-1] * (1 << 15)                   # (rows so wide that a group may be worth a pass of its own)
    wide = most + 6000
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = ints([row[:wide] for row in table])
    T = max(PREFIX, sum(OWN) + 6 * 8)
    meta = layer.StepMeta(T + 64, 1, RANK)
    local, glob = layer.SeqMeta(n, T + 64, wide, HQ, HKV, HD), layer.SeqMeta(n, T + 64, wide, HQ, HKV, HD, max_groups=1)

    def step(rows, lengths, tables, slots, grouped):
        x = torch.cat(rows)
        starts = ints([0] + torch.tensor([len(r) for r in rows]).cumsum(0).tolist())
        most_new = max(len(r) for r in rows)
        meta.build(ints([s for s, r in zip(slots, rows) for _ in range(len(r))]), None, lins[0]["qkv"].pool)
        near = tables.clone()
        for s, L in enumerate(lengths):                 # what has gone out of the window is not looked at
            first = max(0, L - len(rows[s]) - WINDOW + 1)
            near[s, -(-SINKS // PAGE):first // PAGE] = -1
        local.build(starts, ints(lengths), near, len(x), caches[0], most_new, window=WINDOW, sinks=SINKS)
        if grouped:
            glob.build(starts, ints(lengths), tables, len(x), caches[1], most_new, group_start=ints([0, len(rows)]), prefix_len=ints([PREFIX]))
        else:
            glob.build(starts, ints(lengths), tables, len(x), caches[1], most_new)
        for lin, seq, cache in zip(lins, (local, glob), caches):
            y = layer.attention_block(meta, seq, cache, x, lin["qkv"].pool, lin["qkv"].W, lin["o"].pool, lin["o"].W, rope=rope)
            x = (x.float() + y).to(torch.bfloat16)
            y = layer.feed_forward(meta, x, lin["up"].pool, lin["up"].W, lin["down"].pool, lin["down"].W)
            x = (x.float() + y).to(torch.bfloat16)
        for m in (meta, local, glob):
            m.status()
        return x.split([len(r) for r in rows])

    # The prefix, by the base model; its keys and values serve the whole pages for all (its last, partial page is written again by each).
    got_prefix = step([common], [PREFIX], table[:1], [-1], False)[0]
    tail = common[whole * PAGE:]
    out = [[] for _ in range(n)]
    # (the adapters see the tokens behind the prefix's whole pages alone)
    for s, y in enumerate(step([torch.cat((tail, x[:k])) for x, k in zip(own, OWN)], [PREFIX + k for k in OWN], table, slot_of, True)):
        out[s].append(y)
    for i in range(NEW):
        for s, y in enumerate(step([x[k + i:k + i + 1] for x, k in zip(own, OWN)], [PREFIX + k + i + 1 for k in OWN], table, slot_of, True)):
            out[s].append(y)

    def exact(s, bf, kv):
        """Sequence s: base model up to the shared pages' end, its adapter from there on."""
        x = torch.cat((common, own[s])).double()
        cut = whole * PAGE
        for lin, window in zip(lins, (True, False)):
            class Mixed:
                def __init__(self, one):
                    self.one = one

                def exact(self, rows, slot):
                    return torch.cat((self.one.exact(rows[:cut], -1), self.one.exact(rows[cut:], slot)))
            x = exact_block(x, slot_of[s], {k: Mixed(one) for k, one in lin.items()}, window, rope, bf, kv)
        return x[cut:]

    def off_by(most):
        return lambda y: y * (1 + most * (2 * torch.rand(y.shape, generator=g, device="cuda", dtype=torch.float64) - 1))

    nearest = lambda y: y.to(torch.bfloat16).double()  # noqa: E731

    def nearest_e4m3(y):
        scale = y.abs().amax(-1, keepdim=True) / 448
        return (y / scale).float().to(torch.float8_e4m3fn).double() * scale

    some = off_by(2.0 ** -8)
    some_kv = some if kind == "bf16" else off_by(2.0 ** -4)
    for s in range(n):
        got, want = torch.cat(out[s]).double(), exact(s, nearest, nearest if kind == "bf16" else nearest_e4m3)
        noise = torch.stack([(exact(s, some, some_kv) - want).norm(dim=1) for _ in range(8)]).amax(0)
        error, size = (got - want).norm(dim=1), want.norm(dim=1)
        assert (error <= 4 * noise + 2.0 ** -6 * size).all(), (s, (error / (4 * noise + 2.0 ** -6 * size)).tolist())
        assert float(error.median()) < 2 * float(noise.median()) + 2.0 ** -6 * float(size.median())
    assert got_prefix.isfinite().all()
