"""The rest of a served decoder layer: what is measured, over which sizes.

Three operators beside the attention step and the adapted linears:

  window  causal attention of a step's new tokens over the paged cache in which a token sees the last `window` positions (its
          own among them) and the first `sinks` ones; pages that no new token sees have been given back (page -1);
  shared  causal attention of a step in which groups of sequences begin with the same cached tokens (the same pages): the
          shared keys meet the whole group's queries at once;
  gated   the adapted gate_up linear with its activation: h = act(g) * u in bf16, the down linear's input, where
          [g u] = x W^T + sum_j s c B (A x) is the multi-LoRA linear.

`run` computes a case in plain torch operations, or, where `own` is true, through this repository's entry points.
A step's metadata (page tables, work split, slot sort) serves every layer of a step, so `prepare` keeps it, as a serving loop
does; the cases with "build" true build it in the pass, as the step's first layer does.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------- the cases
def _attn(name, op, seqs, new, ctx, hq=32, hkv=8, hd=128, page=16, kind="bf16", **more):
    """new and ctx: "lo-hi" bounds of the new tokens and of the earlier cached tokens of each sequence; shared: ctx are the
    cached tokens behind the prefix, prefix the bounds of the groups' prefixes (the sequences are spread evenly over the groups)."""
    c = {"name": name, "op": op, "seqs": seqs, "new": new, "ctx": ctx, "hq": hq, "hkv": hkv, "hd": hd, "page": page, "kind": kind,
         "chunks": 0, "chunk": 0, "window": 0, "sinks": 0, "groups": 0, "prefix": "0-0", "build": False}
    c.update(more)
    return c


def _gated(name, tokens, K, F, slots, rank, act="silu", J=1, build=False):
    """slots adapters of a rank up to `rank` each, the tokens' slots uniform over them and -1 (no adapter)."""
    return {"name": name, "op": "gated", "tokens": tokens, "K": K, "F": F, "slots": slots, "rank": rank, "act": act, "J": J,
            "build": build}


def listed():
    return [
        # one user's next token far into a conversation, a local layer: latency
        _attn("window_one_token", "window", 1, "1-1", "5000-5000", window=1024, sinks=4),
        # the decode workload's 256 tokens in a local layer, contexts shorter and far longer than the window
        _attn("window_decode_256", "window", 256, "1-1", "200-30000", window=1024, sinks=4),
        # the same over the quantised cache, a wide window that is no multiple of anything, more first tokens
        _attn("window_decode_64_e4m3", "window", 64, "1-1", "2000-120000", page=32, kind="e4m3", window=4001, sinks=70),
        # a long prompt in one piece
        _attn("window_prompt_8000", "window", 1, "8000-8000", "0-0", page=128, window=1024, sinks=4),
        # the mixed serving step: decode tokens and chunks of prompts on top of earlier chunks
        _attn("window_mixed_e4m3", "window", 256, "1-1", "100-9000", page=32, kind="e4m3", chunks=4, chunk=192, window=500, sinks=16,
              build=True),
        # a few continuations of one conversation: latency
        _attn("shared_four", "shared", 4, "1-1", "20-60", groups=1, prefix="1000-1000"),
        # the decode workload behind one system prompt
        _attn("shared_decode_256", "shared", 256, "1-1", "10-500", page=32, groups=1, prefix="4100-4100"),
        # the same, each tenant's sequences behind a prompt of its own, quantised cache
        _attn("shared_tenants_e4m3", "shared", 200, "1-1", "10-800", page=32, kind="e4m3", groups=7, prefix="300-6000", build=True),
        # questions about one document, their prompts in one step
        _attn("shared_prompts", "shared", 16, "50-300", "0-0", page=64, groups=1, prefix="9000-9000"),
        # one user's next token through the mixed step's gate_up linear: the weights' bytes
        _gated("gated_one_token", 1, 4096, 14336, 16, 16),
        # 256 decode tokens of many tenants, metadata built
        _gated("gated_decode_256", 256, 4096, 14336, 100, 16, build=True),
        # the prefill workload's 4096 tokens through gate_up
        _gated("gated_prompts_4096", 4096, 4096, 14336, 8, 64),
    ]


HEADS = [(32, 8, 128), (32, 8, 128), (32, 32, 128), (16, 2, 128), (20, 4, 64), (8, 8, 64), (28, 4, 128), (12, 12, 64),
         (16, 1, 128), (32, 8, 64)]
ACTS = ["silu", "silu", "gelu_tanh", "gelu"]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["window", "window", "shared", "shared", "gated", "gated"])
    if op == "gated":
        return _gated("", _spread(rng, 1, 4096), 8 * _spread(rng, 16, 1100), 8 * _spread(rng, 8, 1792), _spread(rng, 1, 128),
                      rng.choice([8, 16, 40, 64]), rng.choice(ACTS), rng.choice([1, 1, 2, 3]), rng.random() < 0.3)
    hq, hkv, hd = rng.choice(HEADS)
    more = {"hq": hq, "hkv": hkv, "hd": hd, "page": rng.choice([8, 16, 32, 64, 128, 256]), "kind": rng.choice(["bf16", "e4m3"]),
            "build": rng.random() < 0.3}
    form = rng.choice(["decode", "decode", "chunk", "prompt", "mixed"])
    if op == "window":
        more.update(window=_spread(rng, 20, 8000), sinks=rng.choice([0, 1, 4, 4, 64, rng.randint(2, 300)]))
        if form == "decode":
            new, ctx = rng.choice([1, 1, 1, 2, 3]), _spread(rng, 8, 131000)
            return _attn("", op, _spread(rng, 1, 256), "1-%d" % new, "%d-%d" % (ctx // 4, ctx), **more)
        if form == "chunk":
            new, ctx = _spread(rng, 5, 2048), _spread(rng, 8, 32000)
            return _attn("", op, _spread(rng, 1, 16), "%d-%d" % (max(1, new // 2), new), "%d-%d" % (ctx // 4, ctx), **more)
        if form == "prompt":
            new = _spread(rng, 5, 8000)
            return _attn("", op, _spread(rng, 1, 16), "%d-%d" % (max(1, new // 2), new), "0-0", **more)
        return _attn("", op, _spread(rng, 4, 200), "1-1", "10-%d" % _spread(rng, 20, 20000), chunks=rng.choice([1, 2, 4, 7]),
                     chunk=_spread(rng, 10, 300), **more)
    prefix = _spread(rng, 40, 20000)
    more["prefix"] = "%d-%d" % (prefix // 2, prefix)
    if form in ("decode", "mixed"):
        seqs, new = _spread(rng, 2, 256), rng.choice([1, 1, 1, 2, 3])
        return _attn("", op, seqs, "1-%d" % new, "0-%d" % _spread(rng, 5, 1000), groups=rng.randint(1, max(1, min(seqs // 2, 12))),
                     **more)
    seqs, new = _spread(rng, 2, 16), _spread(rng, 5, 500)
    return _attn("", op, seqs, "%d-%d" % (max(1, new // 2), new), "0-%d" % rng.choice([0, 100]),
                 groups=rng.randint(1, max(1, seqs // 2)), **more)


def draw(rng):
    """Another case of these ranges that costs no more than the largest listed ones."""
    while True:
        c = _draw(rng)
        w = work(c)
        if c["op"] == "gated":
            fits = w["flops"] <= 9.8e11 and c["tokens"] * c["F"] <= 6e7
        else:
            n, l = _lengths(c)
            span = max(l) if c["op"] == "shared" else min(max(l), c["sinks"] + c["window"] + max(n))
            cells = len(n) * c["hq"] * max(n) * (span + c["page"])
            keys = len(n) * c["hkv"] * c["hd"] * (span + c["page"])
            fits = w["bytes"] <= 2.0e9 and w["flops"] <= 5.0e11 and cells <= 2.6e9 and keys <= 1.1e9
        if fits:
            del c["name"]
            return c


# ------------------------------------------------------------------------------------------- sizes
def _bounds(text):
    lo, hi = text.split("-")
    return int(lo), int(hi)


def _groups(case):
    """First sequence of each group, and their number at the end; and the groups' prefixes, whole pages: by the case alone."""
    rng = random.Random("%(seqs)d %(groups)d %(prefix)s %(hq)d" % case)
    G, page = case["groups"], case["page"]
    return [case["seqs"] * g // max(G, 1) for g in range(G + 1)], [rng.randint(*_bounds(case["prefix"])) // page * page for _ in range(G)]


def _lengths(case):
    """New tokens and cached length (prefix and new ones among it) of each sequence: by the case alone."""
    rng = random.Random("%(seqs)d %(new)s %(ctx)s %(hq)d %(page)d %(chunks)d %(chunk)d" % case)
    (n0, n1), (c0, c1) = _bounds(case["new"]), _bounds(case["ctx"])
    n = [rng.randint(n0, n1) for _ in range(case["seqs"])] + [case["chunk"]] * case["chunks"]
    l = [k + rng.randint(c0, c1) for k in n]
    order = list(range(len(n)))
    rng.shuffle(order)                     # chunks sit anywhere among the decode tokens
    n, l = [n[i] for i in order], [l[i] for i in order]
    first, prefix = _groups(case)
    for g, p in enumerate(prefix):
        for s in range(first[g], first[g + 1]):
            l[s] += p
    return n, l


def _kept(case, n, L):
    """The first position behind the sinks that some new token of a sequence sees."""
    return max(0, L - n - case["window"] + 1)


def work(case):
    if case["op"] == "gated":
        T, K, F = case["tokens"], case["K"], case["F"]
        slots, ranks = _slots(case)
        used = {s for row in slots for s in row if s >= 0}
        active = sum(ranks[s] for row in slots for s in row if s >= 0)
        return {"bytes": 2 * (T * K + 2 * F * K + T * F + sum(ranks[s] for s in used) * (K + 2 * F)),
                "flops": 4 * T * K * F + 2 * active * (K + 2 * F)}
    n, l = _lengths(case)
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    row = hd * 2 if case["kind"] == "bf16" else hd + 4       # bytes of one cached key or value row
    if case["op"] == "window":
        w, sinks = case["window"], case["sinks"]
        seen = rows = 0
        for k, L in zip(n, l):
            rows += L - _kept(case, k, L) + min(sinks, _kept(case, k, L))
            for p in range(L - k, L):
                lo = max(0, p - w + 1)
                seen += p + 1 - lo + min(sinks, lo)
    else:
        first, prefix = _groups(case)
        seen = sum(k * (b - k) + k * (k + 1) // 2 for k, b in zip(n, l))
        rows = sum(l) - sum(p * (first[g + 1] - first[g] - 1) for g, p in enumerate(prefix))
    return {"bytes": rows * hkv * 2 * row + 2 * sum(n) * hq * hd * 2, "flops": 4 * hd * hq * seen}


# ------------------------------------------------------------------------------------------- inputs
def _tables(case, n, l):
    """Pages of each sequence in the order in which their numbers are handed out, -1 where none is held; and how many."""
    page, rows, used = case["page"], [], 0
    first, prefix = _groups(case)
    group = {s: g for g in range(case["groups"]) for s in range(first[g], first[g + 1])}
    common = {}
    for s, (k, L) in enumerate(zip(n, l)):
        count, row = -(-L // page), []
        g = group.get(s)
        if g is not None:
            whole = prefix[g] // page                       # held once for the group
            if g not in common:
                common[g] = list(range(used, used + whole))
                used += whole
            row = list(common[g])
        for i in range(len(row), count):
            hidden = case["op"] == "window" and i * page >= case["sinks"] and (i + 1) * page <= _kept(case, k, L)
            row.append(-1 if hidden else used)
            used += not hidden
        rows.append(row)
    return rows, used


def _attention_inputs(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *shape, dtype=torch.float32: torch.randn(*shape, generator=g, device=dev, dtype=dtype)  # noqa: E731
    n, l = _lengths(case)
    hq, hkv, hd, page = case["hq"], case["hkv"], case["hd"], case["page"]
    rows, used = _tables(case, n, l)
    n_pages = used + 3
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    most = max(map(len, rows))
    at = torch.tensor([r + [-1] * (most - len(r)) for r in rows], device=dev)
    pages = torch.where(at >= 0, perm[at.clamp(min=0)], torch.full_like(perm[:1], -1))
    first, prefix = _groups(case)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": case, "S": len(n), "T": sum(n), "max_new": max(n), "max_len": max(l), "n_pages": n_pages, "pages": pages.contiguous(),
         "q_start": ints([0] + torch.tensor(n).cumsum(0).tolist()), "kv_len": ints(l),
         "group_start": ints(first), "prefix_len": ints(prefix),
         # what the scheduler that formed the groups knows on the host
         "groups": [(first[i], first[i + 1], p) for i, p in enumerate(prefix)]}
    # keys with a few strong channels, as trained models have them
    gain = torch.exp(0.5 * normal(hkv, 1, hd))
    k = normal(n_pages, hkv, page, hd, dtype=torch.bfloat16).mul_(gain.to(torch.bfloat16))
    v = normal(n_pages, hkv, page, hd, dtype=torch.bfloat16)
    if case["kind"] == "bf16":
        s.update(k=k, v=v, k_scale=None, v_scale=None)
    else:
        for name, x in (("k", k), ("v", v)):
            scale = x.abs().amax(-1).float() / E4M3_MAX
            s[name] = (x.float() / scale[..., None]).to(torch.float8_e4m3fn)
            s[name + "_scale"] = scale
    s["q"] = normal(s["T"], hq, hd, dtype=torch.bfloat16)
    return s


def _slots(case):
    """Slots of each token and the adapters' ranks: by the case alone."""
    rng = random.Random("%(tokens)d %(K)d %(F)d %(slots)d %(rank)d %(J)d" % case)
    ranks = [rng.choice([r for r in (case["rank"], case["rank"] // 2, 8) if r >= 8]) for _ in range(case["slots"])]
    return [[rng.randint(-1, case["slots"] - 1) for _ in range(case["J"])] for _ in range(case["tokens"])], ranks


def _gated_inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape, std=1.0: torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(std)  # noqa: E731
    T, K, F = case["tokens"], case["K"], case["F"]
    slots, ranks = _slots(case)
    scales = 0.2 + 0.8 * torch.rand(T, case["J"], generator=g, device="cuda") if case["J"] > 1 else None
    return {"case": case, "x": rand(T, K), "W": rand(2 * F, K, std=0.02), "slots": torch.tensor(slots, dtype=torch.int32, device="cuda"),
            "scales": scales, "ranks": ranks, "A": [rand(r, K, std=0.02) for r in ranks], "B": [rand(2 * F, r, std=0.02) for r in ranks]}


def _inputs(case, seed):
    return (_gated_inputs if case["op"] == "gated" else _attention_inputs)(case, seed)


ALPHA = 32.0


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from rank_adapter_gemm_token_gb300 import layer
    if case["op"] == "gated":
        T, K, F = case["tokens"], case["K"], case["F"]
        s["pool"] = layer.AdapterPool(case["slots"], case["rank"], K, 2 * F)
        for i, r in enumerate(s["ranks"]):
            s["pool"].load(i, s["A"][i], s["B"][i], r, ALPHA)
        s["pool"].sync()
        s["meta"] = layer.StepMeta(T, case["J"], case["rank"])
        s["meta"].build(s["slots"], s["scales"], s["pool"])
        return s
    hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
    s["cache"] = layer.KVCache(s["n_pages"], case["page"], hkv, hd, k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    s["seq"] = layer.SeqMeta(s["S"], s["T"], s["pages"].shape[1], hq, hkv, hd, max_groups=case["groups"])
    _build(s)
    return s


def _build(s):
    more = ({"window": s["case"]["window"], "sinks": s["case"]["sinks"]} if s["case"]["op"] == "window" else
            {"group_start": s["group_start"], "prefix_len": s["prefix_len"]})
    s["seq"].build(s["q_start"], s["kv_len"], s["pages"], s["T"], s["cache"], max_new=s["max_new"], **more)


# ------------------------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else {"window": _window, "shared": _shared, "gated": _plain_gated}[s["case"]["op"]])(s)


def _run_own(s):
    from rank_adapter_gemm_token_gb300 import layer
    if s["case"]["op"] == "gated":
        if s["case"]["build"]:
            s["meta"].build(s["slots"], s["scales"], s["pool"])
        return layer.gated_linear(s["pool"], s["meta"], s["x"], s["W"], act=s["case"]["act"])
    if s["case"]["build"]:
        _build(s)
    return layer.attention(s["cache"], s["seq"], s["q"])


def _rows(s, x, scale, page, off):
    """Cached rows at (page, offset) [S, keys]: fp32 [S, Hkv, keys, hd]."""
    if scale is None:
        return x[page, :, off].float().transpose(1, 2)
    codes = x.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float()
    return (codes * scale[page, :, off][..., None]).transpose(1, 2)


def _padded_queries(s):
    """Queries [S, Hkv, group, most, hd], and the tokens' sequences and places among their sequence's new tokens."""
    hq, hkv, hd = s["case"]["hq"], s["case"]["hkv"], s["case"]["hd"]
    start = s["q_start"].long()
    i = torch.arange(s["max_new"], device=start.device)
    row = (start[:-1, None] + i).clamp(max=s["T"] - 1)
    q = s["q"][row].float().view(s["S"], s["max_new"], hkv, hq // hkv, hd).permute(0, 2, 3, 1, 4)
    t = torch.arange(s["T"], device=start.device)
    seq = torch.searchsorted(start, t, right=True) - 1
    return q, seq, t - start[seq]


def _window(s):
    c = s["case"]
    hq, hkv, hd, S, window, sinks = c["hq"], c["hkv"], c["hd"], s["S"], c["window"], c["sinks"]
    start, length = s["q_start"].long(), s["kv_len"].long()
    n, most = start[1:] - start[:-1], s["max_new"]
    # positions to look at: the first ones, then those from where the first new token's window begins
    kept = (length - n - window + 1).clamp(min=0)
    head, span = min(sinks, s["max_len"]), min(s["max_len"], window + most - 1)
    at = torch.cat((torch.arange(head, device=n.device).expand(S, head), kept[:, None] + torch.arange(span, device=n.device)), 1)
    double = torch.arange(head + span, device=n.device)[None] >= head                # a first token once more in the window
    held = (at < length[:, None]) & ~(double & (at < sinks))
    page = s["pages"].long().gather(1, (at // c["page"]).clamp(max=s["pages"].shape[1] - 1)).clamp(min=0)
    k, v = (_rows(s, s[x], s[x + "_scale"], page, at % c["page"]) for x in ("k", "v"))
    q, seq, place = _padded_queries(s)
    score = (q.reshape(S, hkv, -1, hd) @ k.transpose(2, 3)).mul_(1 / math.sqrt(hd)).view(S, hkv, hq // hkv, most, -1)
    pos = (length - n)[:, None, None] + torch.arange(most, device=n.device)[:, None]  # [S, most, 1]
    seen = held[:, None] & (at[:, None] <= pos) & ((at[:, None] < sinks) | (at[:, None] > pos - window))
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1, keepdim=True)
    o = ((score.view(S, hkv, -1, score.shape[-1]) @ v).view(S, hkv, hq // hkv, most, hd) / total).permute(0, 3, 1, 2, 4)
    return o.reshape(S, most, hq, hd)[seq, place].to(torch.bfloat16).view(s["T"], hq * hd)


def _shared(s):
    c = s["case"]
    hq, hkv, hd, S, size = c["hq"], c["hkv"], c["hd"], s["S"], c["page"]
    start, length = s["q_start"].long(), s["kv_len"].long()
    n, most = start[1:] - start[:-1], s["max_new"]
    q, seq, place = _padded_queries(s)
    out = torch.empty(S, most, hq, hd, device=n.device)
    i = torch.arange(most, device=n.device)
    for a, b, prefix in s["groups"]:
        m = b - a
        # the prefix's keys once, against all rows of the group; then each sequence's own
        at = torch.arange(prefix, device=n.device)
        kp, vp = (_rows(s, s[x], s[x + "_scale"], s["pages"][a, at // size].long()[None], (at % size)[None])[0] for x in ("k", "v"))
        rest = s["max_len"] - prefix
        at = prefix + torch.arange(rest, device=n.device).expand(m, rest)
        page = s["pages"][a:b].long().gather(1, (at // size).clamp(max=s["pages"].shape[1] - 1)).clamp(min=0)
        k, v = (_rows(s, s[x], s[x + "_scale"], page, at % size) for x in ("k", "v"))
        qg, rows = q[a:b], hq // hkv * most
        zp = (qg.permute(1, 0, 2, 3, 4).reshape(hkv, -1, hd) @ kp.transpose(1, 2)).mul_(1 / math.sqrt(hd))
        zp = zp.view(hkv, m, rows, prefix).transpose(0, 1)
        zs = (qg.reshape(m, hkv, -1, hd) @ k.transpose(2, 3)).mul_(1 / math.sqrt(hd)).view(m, hkv, hq // hkv, most, rest)
        last = (length - n)[a:b, None] + i
        zs.masked_fill_((at[:, None] > last[:, :, None])[:, None, None], float("-inf"))
        zs = zs.view(m, hkv, rows, rest)
        top = zs.amax(-1, keepdim=True)
        if prefix:
            top = torch.maximum(top, zp.amax(-1, keepdim=True))
        zp, zs = (zp - top).exp_(), (zs - top).exp_()
        total = zp.sum(-1, keepdim=True) + zs.sum(-1, keepdim=True)
        o = (zp.transpose(0, 1).reshape(hkv, m * rows, prefix) @ vp).view(hkv, m, rows, hd).transpose(0, 1) + zs @ v
        out[a:b] = (o / total).view(m, hkv, hq // hkv, most, hd).permute(0, 3, 1, 2, 4).reshape(m, most, hq, hd)
    return out[seq, place].to(torch.bfloat16).view(s["T"], hq * hd)


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _plain_gated(s):
    c = s["case"]
    x = s["x"].float()
    y = x @ s["W"].float().T
    # every token against every adapter's rows, what is not its own struck out
    A, B = torch.cat(s["A"]).float(), torch.cat(s["B"], 1).float()
    rank = torch.tensor(s["ranks"], device="cuda")
    owner = torch.repeat_interleave(torch.arange(c["slots"], device="cuda"), rank)
    share = torch.zeros(c["tokens"], len(owner), device="cuda")
    for j in range(c["J"]):
        mine = (s["slots"][:, j:j + 1] == owner).float()
        share += mine if s["scales"] is None else mine * s["scales"][:, j:j + 1]
    y += (x @ A.T * share * (ALPHA / rank[owner])) @ B.T
    g, u = y.split(c["F"], 1)
    return (_act(g, c["act"]) * u).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "gated":
        T, F = case["tokens"], case["F"]
        h = torch.empty(T, F, dtype=torch.float64, device="cuda")
        x = s["x"].double()
        y = torch.cat([x @ w.double().T for w in s["W"].split(4096)], 1)
        slots = s["slots"].cpu()
        for i, r in enumerate(s["ranks"]):
            for j in range(case["J"]):
                rows = torch.nonzero(slots[:, j] == i)[:, 0].cuda()
                if len(rows):
                    d = (x[rows] @ s["A"][i].double().T) @ s["B"][i].double().T * (ALPHA / r)
                    y[rows] += d if s["scales"] is None else d * s["scales"][rows, j:j + 1].double()
        g, u = y[:, :F], y[:, F:]
        if case["act"] == "silu":
            h = g * torch.sigmoid(g)
        elif case["act"] == "gelu_tanh":
            h = g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
        else:
            h = 0.5 * g * torch.special.erfc(-g / math.sqrt(2))
        return h * u
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    hq, hkv, hd, size = case["hq"], case["hkv"], case["hd"], case["page"]
    out = torch.zeros(s["T"], hq, hd, dtype=torch.float64, device="cuda")
    for b in range(s["S"]):
        a, e, L = starts[b], starts[b + 1], lens[b]
        at = torch.arange(L, device="cuda")
        if case["op"] == "window":
            at = at[(at < case["sinks"]) | (at >= _kept(case, e - a, L))]
        page = s["pages"][b, at // size].long()

        def rows(name):
            x = s[name][page, :, at % size] if s[name + "_scale"] is None else (
                s[name].view(torch.uint8)[page, :, at % size].view(torch.float8_e4m3fn))
            return x.double() if s[name + "_scale"] is None else x.double() * s[name + "_scale"][page, :, at % size].double()[..., None]

        k, v = rows("k").transpose(0, 1), rows("v").transpose(0, 1)          # [Hkv, keys, hd]
        for r in range(a, e, 1024):
            t = torch.arange(r, min(e, r + 1024), device="cuda")
            p = (t - e + L)[:, None]
            hide = at[None] > p
            if case["op"] == "window":
                hide |= (at[None] >= case["sinks"]) & (at[None] <= p - case["window"])
            for h in range(hkv):
                heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
                z = torch.einsum("thd,kd->thk", s["q"][t, heads].double(), k[h]) * hd ** -0.5
                out[t, heads] = torch.softmax(z.masked_fill(hide[:, None], -math.inf), 2) @ v[h]
    return out.view(s["T"], hq * hd)
