"""The attention step around the multi-LoRA linears: what is measured, over which sizes.

Three operators stand between the qkv linear's fp32 output and the o linear's bf16 input:

  write   the qkv rows of a step: RMS norm of each query and key head, rotary positions, queries rounded to
          bf16, keys and values written to the pages of a paged cache (bf16, or e4m3 with one fp32 scale for
          each token and head);
  attend  causal attention of a step's new tokens (one per sequence, a chunk, or a whole prompt, packed one
          sequence after another) over the paged cache, grouped heads;
  read    the cached keys and values of whole sequences read back as dense bf16 rows.

`run` computes a case in plain torch operations, or, where `own` is true, through this repository's entry points.
A sequence's step metadata (page table checks, work split) serves every layer of a step, so `prepare` keeps it, as
a serving loop does; the cases with "build" true build it in the pass, as the step's first layer does.
"""
import math
import random

import torch

own = False

THETA = 10000.0
EPS = 1e-6
AMAX_MIN = 2.0 ** -60          # rows below this magnitude quantise against it
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------- the cases
def _case(name, op, seqs, new, ctx, hq=32, hkv=8, hd=128, page=16, kind="bf16", **more):
    """new and ctx: "lo-hi" bounds of the new tokens and of the earlier cached tokens of each sequence."""
    c = {"name": name, "op": op, "seqs": seqs, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "hd": hd, "page": page,
         "kind": kind, "chunks": 0, "chunk": 0, "norm": False, "rot": hd, "inter": False, "build": False}
    c.update(more)
    return c


def listed():
    return [
        # one user's next token, right after the qkv linear: latency
        _case("write_one_token", "write", 1, "1-1", "700-700", norm=True),
        # the decode workload's 256 tokens (qkv 4096 -> 6144: 32 query and 8 key/value heads of 128)
        _case("write_decode_256", "write", 256, "1-1", "64-1500", norm=True),
        # the prefill workload's 8 x 512 prompt tokens, quantised as they are written, interleaved partial rotation
        _case("write_prompts_e4m3", "write", 8, "512-512", "0-0", page=64, kind="e4m3", rot=64, inter=True),
        # one user's next token over a short conversation: latency
        _case("attend_one_token", "attend", 1, "1-1", "500-500"),
        # the decode workload: 256 sequences, ragged contexts
        _case("attend_decode_256", "attend", 256, "1-1", "200-2000"),
        # the same with the quantised cache
        _case("attend_decode_256_e4m3", "attend", 256, "1-1", "200-2000", page=32, kind="e4m3"),
        # one user's next token over a long document: the key axis has to be split
        _case("attend_long_context", "attend", 1, "1-1", "131000-131000", page=64),
        # the prefill workload: 8 prompts of 512 tokens
        _case("attend_prompts_8x512", "attend", 8, "512-512", "0-0", page=64),
        # one long prompt in one piece
        _case("attend_prompt_8000", "attend", 1, "8000-8000", "0-0", page=128),
        # the mixed serving step: 256 decode tokens and 4 chunks of 192 tokens on top of earlier chunks
        _case("attend_mixed_e4m3", "attend", 256, "1-1", "100-1500", page=32, kind="e4m3", chunks=4, chunk=192, build=True),
        # a sequence handed to another holder of caches: short, plain
        _case("read_one", "read", 1, "1-1", "1000-1000"),
        # the preempted sequences of a step, quantised cache
        _case("read_batch_e4m3", "read", 16, "1-1", "500-8000", page=32, kind="e4m3"),
    ]


HEADS = [(32, 8, 128), (32, 8, 128), (32, 32, 128), (16, 2, 128), (20, 4, 64), (8, 8, 64), (28, 4, 128), (12, 12, 64),
         (16, 1, 128), (32, 8, 64)]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend", "read"])
    hq, hkv, hd = rng.choice(HEADS)
    more = {"hq": hq, "hkv": hkv, "hd": hd, "page": rng.choice([8, 16, 32, 64, 128, 256]), "kind": rng.choice(["bf16", "e4m3"])}
    if op == "write":
        seqs = _spread(rng, 1, 256)
        new = _spread(rng, 1, 4096 // seqs)
        more.update(norm=rng.random() < 0.5, rot=rng.choice([hd, hd // 2, 24]), inter=rng.random() < 0.5)
        return _case("", op, seqs, "%d-%d" % (max(1, new // 2), new), "0-%d" % rng.choice([0, 100, 3000]), **more)
    if op == "read":
        seqs, ctx = _spread(rng, 1, 32), _spread(rng, 1, 8000)
        return _case("", op, seqs, "1-1", "%d-%d" % (ctx // 3, ctx), **more)
    form = rng.choice(["decode", "decode", "chunk", "prompt", "mixed"])
    if form == "decode":
        seqs = _spread(rng, 1, 256)
        new, ctx = rng.choice([1, 1, 1, 2, 3]), _spread(rng, 8, 131000)
        return _case("", op, seqs, "%d-%d" % (1, new), "%d-%d" % (ctx // 4, ctx), **more)
    if form == "chunk":
        new, ctx = _spread(rng, 5, 2048), _spread(rng, 8, 32000)
        return _case("", op, _spread(rng, 1, 16), "%d-%d" % (max(1, new // 2), new), "%d-%d" % (ctx // 4, ctx), **more)
    if form == "prompt":
        new = _spread(rng, 5, 8000)
        return _case("", op, _spread(rng, 1, 16), "%d-%d" % (max(1, new // 2), new), "0-0", **more)
    return _case("", op, _spread(rng, 4, 200), "1-1", "10-%d" % _spread(rng, 20, 2000), chunks=rng.choice([1, 2, 4, 7]),
                 chunk=_spread(rng, 10, 300), build=True, **more)


def draw(rng):
    """Another case of these ranges that costs no more than the largest listed ones."""
    while True:
        c = _draw(rng)
        w = work(c)
        n, l = _lengths(c)
        cells = len(n) * c["hq"] * max(n) * (max(l) + c["page"])
        keys = len(n) * c["hkv"] * c["hd"] * (max(l) + c["page"])
        if w["bytes"] <= 2.0e9 and w["flops"] <= 5.0e11 and cells <= 2.6e9 and keys <= 1.1e9:
            del c["name"]
            return c


# ------------------------------------------------------------------------------------------- sizes
def _bounds(text):
    lo, hi = text.split("-")
    return int(lo), int(hi)


def _lengths(case):
    """New tokens and cached length (new ones among it) of each sequence: by the case alone."""
    rng = random.Random("%(seqs)d %(new)s %(ctx)s %(hq)d %(page)d %(chunks)d %(chunk)d" % case)
    (n0, n1), (c0, c1) = _bounds(case["new"]), _bounds(case["ctx"])
    n = [rng.randint(n0, n1) for _ in range(case["seqs"])] + [case["chunk"]] * case["chunks"]
    l = [k + rng.randint(c0, c1) for k in n]
    order = list(range(len(n)))
    rng.shuffle(order)                     # chunks sit anywhere among the decode tokens
    return [n[i] for i in order], [l[i] for i in order]


def work(case):
    n, l = _lengths(case)
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    T = sum(n)
    row = hd * 2 if case["kind"] == "bf16" else hd + 4       # bytes of one cached key or value row
    if case["op"] == "write":
        return {"bytes": T * ((hq + 2 * hkv) * hd * 4 + hq * hd * 2 + 2 * hkv * row), "flops": T * (hq + hkv) * hd * 6}
    if case["op"] == "read":
        return {"bytes": sum(l) * hkv * 2 * (row + hd * 2), "flops": sum(l) * hkv * hd * 2}
    seen = sum(k * (b - k) + k * (k + 1) // 2 for k, b in zip(n, l))
    return {"bytes": sum(l) * hkv * 2 * row + 2 * T * hq * hd * 2, "flops": 4 * hd * hq * seen}


# ------------------------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *shape, dtype=torch.float32: torch.randn(*shape, generator=g, device=dev, dtype=dtype)  # noqa: E731
    n, l = _lengths(case)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    S, T = len(n), sum(n)
    most = max(-(-x // page) for x in l)
    used = sum(-(-x // page) for x in l)
    n_pages = used + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    counts = torch.tensor([-(-x // page) for x in l], device=dev)
    at = torch.arange(most, device=dev)[None, :]
    first = (torch.cumsum(counts, 0) - counts)[:, None]
    pages = torch.where(at < counts[:, None], perm[(first + at).clamp(max=n_pages - 1)], torch.full_like(perm[:1], -1))
    s = {"case": case, "S": S, "T": T, "max_new": max(n), "max_len": max(l), "n_pages": n_pages,
         "pages": pages.contiguous(),
         "q_start": torch.tensor([0] + torch.tensor(n).cumsum(0).tolist(), dtype=torch.int32, device=dev),
         "kv_len": torch.tensor(l, dtype=torch.int32, device=dev)}
    # keys with a few strong channels, as trained models have them
    gain = torch.exp(0.5 * normal(hkv, 1, hd))
    k = normal(n_pages, hkv, page, hd, dtype=torch.bfloat16).mul_(gain.to(torch.bfloat16))
    v = normal(n_pages, hkv, page, hd, dtype=torch.bfloat16)
    if case["op"] == "write":              # a new cache: what comes back beside zeros is what was written
        k.zero_(), v.zero_()
    if case["kind"] == "bf16":
        s.update(k=k, v=v, k_scale=None, v_scale=None)
    else:
        for name, x in (("k", k), ("v", v)):
            scale = x.abs().amax(-1).float().clamp(min=AMAX_MIN) / E4M3_MAX
            s[name] = (x.float() / scale[..., None]).to(torch.float8_e4m3fn)
            s[name + "_scale"] = scale
    if case["op"] == "attend":
        s["q"] = normal(T, hq, hd, dtype=torch.bfloat16)
    if case["op"] == "write":
        s["qkv"] = normal(T, (hq + 2 * hkv) * hd)
        s["q_norm"] = (1 + 0.1 * normal(hd)).to(torch.bfloat16) if case["norm"] else None
        s["k_norm"] = (1 + 0.1 * normal(hd)).to(torch.bfloat16) if case["norm"] else None
        pos = torch.arange(max(l), device=dev, dtype=torch.float64)
        freq = THETA ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        s["cos"], s["sin"] = (f(pos[:, None] * freq).float() for f in (torch.cos, torch.sin))
    if case["op"] == "read":
        s["row_start"] = torch.tensor([0] + torch.tensor(l).cumsum(0).tolist(), dtype=torch.int32, device=dev)
        s["rows"] = sum(l)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from rank_adapter_gemm_token_gb300 import layer
        hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
        s["cache"] = layer.KVCache(s["n_pages"], case["page"], hkv, hd, k=s["k"], v=s["v"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
        s["seq"] = layer.SeqMeta(s["S"], s["T"], s["pages"].shape[1], hq, hkv, hd)
        s["seq"].build(s["q_start"], s["kv_len"], s["pages"], s["T"], s["cache"], max_new=s["max_new"])
        if case["op"] == "write":
            s["rope"] = layer.Rope(case["rot"], THETA, interleaved=case["inter"])
    return s


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else {"write": _write, "attend": _attend, "read": _read}[s["case"]["op"]])(s)


def _run_own(s):
    from rank_adapter_gemm_token_gb300 import layer
    if s["case"]["build"]:
        s["seq"].build(s["q_start"], s["kv_len"], s["pages"], s["T"], s["cache"], max_new=s["max_new"])
    op = s["case"]["op"]
    if op == "write":
        q = layer.qkv_write(s["cache"], s["seq"], s["qkv"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, rope=s["rope"])
        return _written(s, q)
    if op == "attend":
        return layer.attention(s["cache"], s["seq"], s["q"])
    return layer.kv_read(s["cache"], s["seq"], s["row_start"], s["rows"])


def _written(s, q):
    out = {"q": q, "k": s["k"], "v": s["v"]}
    if s["k_scale"] is not None:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _tokens(s):
    """Sequence and position of each token."""
    start, length = s["q_start"].long(), s["kv_len"].long()
    t = torch.arange(s["T"], device=start.device)
    seq = torch.searchsorted(start, t, right=True) - 1
    return seq, length[seq] - start[seq + 1] + t


def _rotate(x, cos, sin, rot, inter):
    """x [T, H, hd]: the first rot elements of each head turned by the token's angles [T, rot / 2]."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else r.chunk(2, -1)
    c, d = cos[:, None], sin[:, None]
    p, q = a * c - b * d, b * c + a * d
    turned = torch.stack((p, q), -1).flatten(-2) if inter else torch.cat((p, q), -1)
    return torch.cat((turned, rest), -1)


def _write(s):
    c = s["case"]
    hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
    q, k, v = s["qkv"].view(s["T"], hq + 2 * hkv, hd).split((hq, hkv, hkv), 1)
    if s["q_norm"] is not None:
        q, k = (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
                for x, w in ((q, s["q_norm"]), (k, s["k_norm"])))
    seq, pos = _tokens(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    q, k = (_rotate(x, cos, sin, c["rot"], c["inter"]) for x in (q, k))
    page, off = s["pages"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["kind"] == "bf16":
        s["k"][page, :, off] = k.to(torch.bfloat16)
        s["v"][page, :, off] = v.to(torch.bfloat16)
        return _written(s, q.to(torch.bfloat16))
    k_scale, v_scale = (x.abs().amax(-1).clamp(min=AMAX_MIN) / E4M3_MAX for x in (k, v))
    s["k"].view(torch.uint8)[page, :, off] = (k / k_scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["v"].view(torch.uint8)[page, :, off] = (v / v_scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    s["k_scale"][page, :, off] = k_scale
    s["v_scale"][page, :, off] = v_scale
    return _written(s, q.to(torch.bfloat16))


def _dense(s, x, scale):
    """Cached rows of every sequence, padded to whole pages of the longest: fp32 [S, Hkv, keys, hd]."""
    pages = s["pages"].long().clamp(min=0)
    if scale is None:
        d = x[pages].float()
    else:
        d = x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * scale[pages][..., None]
    S, P, H, size, hd = d.shape
    return d.transpose(1, 2).reshape(S, H, P * size, hd)


def _attend(s):
    c = s["case"]
    hq, hkv, hd, S = c["hq"], c["hkv"], c["hd"], s["S"]
    k, v = _dense(s, s["k"], s["k_scale"]), _dense(s, s["v"], s["v_scale"])
    start, length = s["q_start"].long(), s["kv_len"].long()
    n, most, keys = start[1:] - start[:-1], s["max_new"], k.shape[2]
    i = torch.arange(most, device=k.device)
    row = (start[:-1, None] + i).clamp(max=s["T"] - 1)                                   # [S, most]
    q = s["q"][row].float().view(S, most, hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4).reshape(S, hkv, -1, hd)
    score = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(hd)).view(S, hkv, hq // hkv, most, keys)
    last = length[:, None] - n[:, None] + i                                              # position of each row
    hidden = torch.arange(keys, device=k.device) > last[:, :, None]
    score.masked_fill_(hidden[:, None, None], float("-inf"))
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    o = ((score.view(S, hkv, -1, keys) @ v).view(S, hkv, hq // hkv, most, hd) / total).permute(0, 3, 1, 2, 4)
    seq, pos = _tokens(s)
    t = torch.arange(s["T"], device=k.device)
    return o.reshape(S, most, hq, hd)[seq, t - start[seq]].to(torch.bfloat16).view(s["T"], hq * hd)


def _read(s):
    start, length = s["row_start"].long(), s["kv_len"].long()
    t = torch.arange(s["rows"], device=start.device)
    seq = torch.searchsorted(start, t, right=True) - 1
    pos = t - start[seq]
    page, off = s["pages"][seq, pos // s["case"]["page"]].long(), pos % s["case"]["page"]
    if s["k_scale"] is None:
        return s["k"][page, :, off], s["v"][page, :, off]
    return tuple((x.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float() * z[page, :, off][..., None]).to(torch.bfloat16)
                 for x, z in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    hq, hkv, hd, size = case["hq"], case["hkv"], case["hd"], case["page"]
    group = hq // hkv

    def rows(name, b):
        """Cached rows [L, Hkv, hd] of sequence b."""
        table = s["pages"][b, : -(-lens[b] // size)].tolist()
        x = torch.cat([s[name][p].double() * (1.0 if s[name + "_scale"] is None else s[name + "_scale"][p].double()[..., None])
                       for p in table], 1)
        return x[:, : lens[b]].transpose(0, 1)

    if case["op"] == "read":
        return tuple(torch.cat([rows(name, b) for b in range(s["S"])]) for name in ("k", "v"))
    if case["op"] == "attend":
        out = torch.zeros(s["T"], hq, hd, dtype=torch.float64, device="cuda")
        for b in range(s["S"]):
            k, v = rows("k", b), rows("v", b)
            a, e = starts[b], starts[b + 1]
            for h in range(hq):
                for r in range(a, e, 2048):
                    t = torch.arange(r, min(e, r + 2048), device="cuda")
                    z = s["q"][t, h].double() @ k[:, h // group].T * hd ** -0.5
                    far = torch.arange(lens[b], device="cuda")[None] > (t - e + lens[b])[:, None]
                    out[t, h] = torch.softmax(z.masked_fill(far, -math.inf), 1) @ v[:, h // group]
        return out.view(s["T"], hq * hd)
    # write: heads normalised, turned as complex numbers, then placed
    x = s["qkv"].double().view(s["T"], hq + 2 * hkv, hd)
    pos = torch.cat([torch.arange(lens[b] - (starts[b + 1] - starts[b]), lens[b], device="cuda") for b in range(s["S"])])
    m = case["rot"] // 2
    turn = torch.polar(torch.ones(s["T"], 1, m, dtype=torch.float64, device="cuda"),
                       (pos.double()[:, None] * THETA ** (-torch.arange(m, device="cuda", dtype=torch.float64) / m))[:, None])

    def head(y, w):
        if w is not None:
            y = y / (y.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        y = y.clone()
        one, two = (slice(0, 2 * m, 2), slice(1, 2 * m, 2)) if case["inter"] else (slice(0, m), slice(m, 2 * m))
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y

    q, k, v = head(x[:, :hq], s["q_norm"]), head(x[:, hq:hq + hkv], s["k_norm"]), x[:, hq + hkv:]
    out = {"q": q}
    page = torch.cat([s["pages"][b, torch.arange(lens[b] - (starts[b + 1] - starts[b]), lens[b], device="cuda") // size]
                      for b in range(s["S"])]).long()
    for name, y in (("k", k), ("v", v)):
        kept = s[name].double()
        if case["kind"] == "e4m3":
            scale = y.abs().amax(-1).clamp(min=AMAX_MIN) / E4M3_MAX
            kept_scale = s[name + "_scale"].double()
            kept_scale[page, :, pos % size] = scale
            out[name + "_scale"] = kept_scale
            y = y / scale[..., None]
        kept[page, :, pos % size] = y
        out[name] = kept
    return out
