"""Cases, plain forms and calls of the operators around the verify step.

Four operators of a loop that verifies draft trees over a bounded cache:

* ``encode`` -- RMS norm of each query and key head, the position rotation, and
  the value rows, from a projection's output to what the attention takes; the
  positions are given, or follow from the committed length and the draft tree;
* ``sample`` -- a token from each row of logits by temperature, top-k, top-p and
  min-p and a given random number; over a draft tree also the walk along the
  children that were drawn;
* ``weigh``  -- the attention weight that each cached key receives from the last
  committed rows, added to what it had received before;
* ``evict``  -- the rows of a cache that received the most weight, with the
  first and the latest ones, moved into a smaller cache.

``own = False`` runs the plain forms (elementary torch operations, 32 bits; 64
for angles, running sums of probabilities and what is compared with them);
``own = True`` makes the calls a user makes.
"""

import math

import torch

own = False

DEV = "cuda"
FLOOR = 40           # a token below 2^-FLOOR of the most likely one is never drawn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token over a long context, a quarter of each head rotated
        {"name": "encode_token", "op": "encode", "rows": 1, "hq": 24, "hkv": 4, "d": 256,
         "rot": 64, "pairs": "half", "where": "next", "ctx": 131060, "src": "bf16"},
        # every node of a verify step (budget 22), positions from the tree
        {"name": "encode_tree", "op": "encode", "rows": 23, "hq": 24, "hkv": 4, "d": 256,
         "rot": 256, "pairs": "half", "where": "tree", "ctx": 61440, "src": "bf16"},
        # a prompt of odd length, 32/8 heads of 128, neighbouring dims paired, positions given
        {"name": "encode_prompt", "op": "encode", "rows": 16411, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "pairs": "near", "where": "given", "ctx": 0, "src": "bf16"},
        # one request's next token
        {"name": "sample_token", "op": "sample", "rows": 1, "vocab": 151936, "src": "f32",
         "temperature": 0.8, "top_k": 50, "top_p": 0.95, "min_p": 0.0, "tree": False},
        # every node of a verify step, and the walk
        {"name": "sample_tree", "op": "sample", "rows": 23, "vocab": 151936, "src": "bf16",
         "temperature": 0.7, "top_k": 0, "top_p": 0.9, "min_p": 0.02, "tree": True},
        # a large batch, nucleus sampling
        {"name": "sample_batch", "op": "sample", "rows": 1024, "vocab": 151936, "src": "bf16",
         "temperature": 1.0, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "tree": False},
        # one decoded token over the 128K context
        {"name": "weigh_token_128k", "op": "weigh", "rows": 1, "hq": 24, "hkv": 4, "d": 256,
         "ctx": 131060, "fmt": "q4_0", "window": 0},
        # the accepted nodes of a verify step
        {"name": "weigh_accepted", "op": "weigh", "rows": 9, "hq": 24, "hkv": 4, "d": 256,
         "ctx": 61449, "fmt": "q4_0", "window": 0},
        # the last rows of a prompt in a binary16 cache, heads of 128
        {"name": "weigh_prompt_end", "op": "weigh", "rows": 65, "hq": 32, "hkv": 8, "d": 128,
         "ctx": 32791, "fmt": "f16", "window": 0},
        # a 4096-row cache halved
        {"name": "evict_half", "op": "evict", "hkv": 4, "d": 256, "ctx": 4097, "keep": 2048,
         "sinks": 4, "recent": 256, "fmt": "q4_0"},
        # a binary16 cache with heads of 128 cut to an odd length
        {"name": "evict_f16", "op": "evict", "hkv": 8, "d": 128, "ctx": 61440, "keep": 8191,
         "sinks": 0, "recent": 64, "fmt": "f16"},
        # a 128K prompt cut to a quarter
        {"name": "evict_prompt", "op": "evict", "hkv": 4, "d": 256, "ctx": 131072, "keep": 32768,
         "sinks": 64, "recent": 2048, "fmt": "q4_0"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["encode", "sample", "sample", "weigh", "evict"])
    if op == "sample":
        vocab = _log_int(rng, 33, 151936)
        tree = rng.random() < 0.4
        rows = (rng.randint(1, 65) if tree
                else _log_int(rng, 1, max(1, min(4096, 1024 * 151936 // vocab))))
        return {"op": op, "rows": rows, "vocab": vocab, "tree": tree,
                "src": rng.choice(["bf16", "f32"]) if rows * vocab < 7e7 else "bf16",
                "temperature": rng.choice([1.0, 0.0, round(rng.uniform(0.3, 1.5), 3)]),
                "top_k": rng.choice([0, 0, _log_int(rng, 1, vocab)]),
                "top_p": rng.choice([1.0, round(rng.uniform(0.1, 0.99), 3)]),
                "min_p": rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)])}
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "evict":
        ctx = _log_int(rng, 1, min(131072, 131072 * 4 * 256 // (hkv * d)))
        fmt = rng.choice(["q4_0", "f16"])
        keep = _log_int(rng, 1, max(1, min(ctx, 32768) // (4 if fmt == "f16" else 1)))
        sinks = rng.choice([0, min(keep, rng.randint(1, 64))])
        return {"op": op, "hkv": hkv, "d": d, "ctx": ctx, "keep": keep, "sinks": sinks,
                "recent": rng.choice([0, rng.randint(0, keep - sinks)]), "fmt": fmt}
    hq = hkv * rng.choice([1, 2, 4, 5, 6, 8])
    if op == "encode":
        where = rng.choice(["next", "tree", "given"])
        most = 16411 * 48 * 128 // ((hq + 2 * hkv) * d)
        rows = rng.randint(1, 65) if where == "tree" else _log_int(rng, 1, min(most, 65536))
        return {"op": op, "rows": rows, "hq": hq, "hkv": hkv, "d": d,
                "rot": rng.choice([d, d, d // 2, d // 4]), "pairs": rng.choice(["half", "near"]),
                "where": where, "ctx": _log_int(rng, 1, 131072),
                "src": rng.choice(["bf16", "f32"]) if 2 * rows < most else "bf16"}
    rows = rng.choice([1, rng.randint(2, 17), rng.randint(2, 65)])
    most = min(131072, 131072 * 4 * 256 // (hkv * d),
               int(32791 * 32 * 65 * 128 / (hq * d * rows)))
    ctx = max(rows, _log_int(rng, 1, most))
    fmt = rng.choice(["q4_0", "f16"])
    return {"op": op, "rows": rows, "hq": hq, "hkv": hkv, "d": d,
            "ctx": max(rows, ctx // (2 if fmt == "f16" else 1)), "fmt": fmt,
            "window": rng.choice([0, 0, _log_int(rng, 1, 4096)])}


def _row_bytes(case):
    return case["d"] * 2 if case["fmt"] == "f16" else case["d"] // 32 * 18


def work(case):
    op = case["op"]
    if op == "encode":
        heads, d = case["hq"] + 2 * case["hkv"], case["d"]
        size = 4 if case["src"] == "f32" else 2
        return {"bytes": case["rows"] * heads * d * (size + 2),
                "flops": 8.0 * case["rows"] * (case["hq"] + case["hkv"]) * d}
    if op == "sample":
        size = 4 if case["src"] == "f32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 12),
                "flops": 4.0 * case["rows"] * case["vocab"]}
    if op == "weigh":
        n, ctx = case["rows"], case["ctx"]
        seen = min(ctx, case["window"] + n - 1) if case["window"] else ctx
        return {"bytes": case["hkv"] * (seen * _row_bytes(case) + ctx * 8)
                + n * case["hq"] * (case["d"] * 2 + 4),
                "flops": 2.0 * n * case["hq"] * case["d"] * min(seen, case["window"] or seen)}
    n = min(case["ctx"], case["keep"])
    back = 2 * case["d"] if case["fmt"] == "q4_0" else 0       # rows read back as values
    return {"bytes": case["hkv"] * (case["ctx"] * 4 + n * (4 * _row_bytes(case) + 8 + 2 * back)),
            "flops": 4.0 * case["hkv"] * case["ctx"]}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _floats(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _tree(seed, n):
    """Parents of a random draft tree of n nodes, at most 16 deep."""
    g = torch.Generator()
    g.manual_seed(int(seed) + 17)
    parent, depth = [-1], [0]
    for i in range(1, n):
        p = int(torch.randint(0, i, (1,), generator=g))
        p = p if depth[p] < 16 else 0
        parent.append(p)
        depth.append(depth[p] + 1)
    return torch.tensor(parent, dtype=torch.int32, device=DEV)


def _cache_bytes(g, case):
    """K and V of a filled cache, [hkv, ctx, row bytes]."""
    hkv, ctx, d = case["hkv"], case["ctx"], case["d"]
    out = []
    for _ in range(2):
        if case["fmt"] == "f16":
            x = torch.randn(hkv, ctx, d, generator=g, device=DEV).half()
            out.append(x.view(torch.uint8))
            continue
        # blocks of 32 values: a binary16 scale, then 16 bytes of 4-bit codes
        b = torch.randint(0, 256, (hkv, ctx, d // 32, 18), generator=g, device=DEV,
                          dtype=torch.uint8)
        scale = 0.1 + 0.25 * torch.rand(hkv, ctx, d // 32, 1, generator=g, device=DEV)
        b[..., :2] = scale.half().view(torch.uint8)
        out.append(b.view(hkv, ctx, -1))
    return out


def _values(rows, case, dtype=torch.float32):
    """What cache rows [..., row bytes] stand for, [..., d]."""
    if case["fmt"] == "f16":
        return rows.contiguous().view(torch.float16).to(dtype)
    b = rows.reshape(*rows.shape[:-1], case["d"] // 32, 18)
    scale = b[..., :2].contiguous().view(torch.float16).to(dtype)
    code = torch.cat([b[..., 2:] & 15, b[..., 2:] >> 4], -1).to(dtype) - 8.0
    return (code * scale).reshape(*rows.shape[:-1], case["d"])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "encode":
        n, hq, hkv, d = (case[k] for k in ("rows", "hq", "hkv", "d"))
        # one projection's output: queries, keys and values of a row side by side
        x = torch.randn(n, (hq + 2 * hkv) * d, generator=g, device=DEV).to(_floats(case["src"]))
        s["q"] = x[:, :hq * d].view(n, hq, d)
        s["k"] = x[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
        s["v"] = x[:, (hq + hkv) * d:].view(n, hkv, d)
        s["q_weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["k_weight"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["ctx_len"] = torch.tensor([case["ctx"]], dtype=torch.int32, device=DEV)
        s["dropped"] = torch.randint(0, 4096, (1,), generator=g, device=DEV, dtype=torch.int32)
        if case["where"] == "tree":
            s["parent"] = _tree(seed, n)
        elif case["where"] == "given":
            s["positions"] = torch.randint(0, 131072, (n,), generator=g, device=DEV,
                                           dtype=torch.int32)
        if own:
            from tree_verify_attention_gb300 import api
            s["rope"] = api.Rope(d, case["rot"], base=1e6, interleaved=case["pairs"] == "near",
                                 device=DEV)
            s["out"] = tuple(torch.empty(n, h, d, dtype=torch.bfloat16, device=DEV)
                             for h in (hq, hkv, hkv))
        return s
    if op == "sample":
        n, v = case["rows"], case["vocab"]
        x = torch.randn(n, v, generator=g, device=DEV) * 2.0
        likely = torch.randint(0, v, (n, 24), generator=g, device=DEV)
        # a few plausible tokens in each row, on a model's usual scale
        high = 6.0 + 9.0 * torch.rand(n, 24, generator=g, device=DEV)
        x.scatter_reduce_(1, likely, high, "amax")
        s["logits"] = x.to(_floats(case["src"]))
        s["uniform"] = torch.rand(n, generator=g, device=DEV)
        if case["tree"]:
            s["parent"] = _tree(seed, n)
            best = x.scatter(1, likely[:, :1], 14.0).topk(min(4, v), 1).indices
            pick = torch.randint(0, best.shape[1], (n, 1), generator=g, device=DEV)
            drafted = best[s["parent"].long().clamp(min=0)].gather(1, pick)[:, 0]
            s["tokens"] = drafted.to(torch.int32)
        if own:
            from tree_verify_attention_gb300 import api
            s["sampling"] = api.Sampling(temperature=case["temperature"], top_k=case["top_k"],
                                         top_p=case["top_p"], min_p=case["min_p"])
            s["token"] = torch.empty(n, dtype=torch.int32, device=DEV)
            s["logprob"] = torch.empty(n, device=DEV)
            if case["tree"]:
                s["accept_len"] = torch.empty(1, dtype=torch.int32, device=DEV)
                s["path"], s["out_tokens"] = (torch.empty(n, dtype=torch.int32, device=DEV)
                                              for _ in range(2))
                s["ws"] = api.workspace(api.sample_accept_workspace_bytes(n, v), device=DEV)
        return s
    s["k"], s["v"] = _cache_bytes(g, case)
    hkv, d, ctx = case["hkv"], case["d"], case["ctx"]
    # what the keys have received so far: a few far more than the others
    s["weights"] = torch.exp(2.0 * torch.randn(hkv, ctx, generator=g, device=DEV)) * 1e-3
    if op == "weigh":
        n, hq = case["rows"], case["hq"]
        s["q"] = torch.randn(n, hq, d, generator=g, device=DEV).to(torch.bfloat16)
        x = _scores(s).masked_fill(~_seen(s)[None, :, None, :], -math.inf)
        s["lse"] = torch.logsumexp(x, -1).permute(1, 0, 2).reshape(n, hq).contiguous()
        del x, s["v"]
    if own:
        from tree_verify_attention_gb300 import api
        s["cache"] = _cache(api, case, s, ctx)
        if op == "weigh":
            s["out"] = torch.empty(hkv, ctx, device=DEV)
        else:
            n = min(ctx, case["keep"])
            s["into"] = api.KVCache(hkv, d, n, device=DEV, fmt=case["fmt"])
            s["kept"] = torch.empty(hkv, n, dtype=torch.int32, device=DEV)
            s["weights_out"] = torch.empty(hkv, n, device=DEV)
            s["rows_out"] = tuple(torch.empty(hkv, n, d, dtype=torch.bfloat16, device=DEV)
                                  for _ in range(2))
    return s


def _cache(api, case, s, ctx):
    cache = api.KVCache(case["hkv"], case["d"], ctx, device=DEV, fmt=case["fmt"])
    cache.k.copy_(s.pop("k"))
    if "v" in s:
        cache.v.copy_(s.pop("v"))
    cache.ctx_len.fill_(ctx)
    return cache


# ---------------------------------------------------------------- plain forms

def _ancestors(parent):
    """Ancestor-or-self matrix [n, n] of a tree, from powers of its adjacency."""
    n = parent.numel()
    step = torch.eye(n, dtype=torch.float64, device=parent.device)
    step[torch.arange(1, n, device=parent.device), parent[1:].long()] = 1.0
    return torch.linalg.matrix_power(step, 64) > 0


def _plain_encode(s):
    case = s["case"]
    n, d, rot = case["rows"], case["d"], case["rot"]
    if case["where"] == "given":
        pos = s["positions"].double()
    else:
        step = (_ancestors(s["parent"]).sum(1) - 1 if case["where"] == "tree"
                else torch.arange(n, device=DEV))
        pos = (s["ctx_len"] + s["dropped"] + step).double()
    freq = 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    angle = (pos[:, None] * freq)[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        if case["pairs"] == "near":
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, x[..., rot:]], -1).to(torch.bfloat16)

    return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"]),
            "v": s["v"].to(torch.bfloat16).contiguous()}


def _plain_sample(s):
    case = s["case"]
    x = s["logits"].float()
    n, vocab = x.shape
    m = x.amax(1, keepdim=True)
    # one whole number for each value that orders by value, then by lower index
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32)
    key = key + (vocab - 1 - torch.arange(vocab, device=x.device))
    order = torch.sort(key, 1, descending=True).indices
    if case["temperature"] == 0.0:
        token, logprob = order[:, 0], torch.zeros(n, device=DEV)
    else:
        z = (x.double() - m.double()) / float(torch.tensor(case["temperature"]))
        w = torch.exp(z)
        sw = w.gather(1, order)
        rank = torch.arange(vocab, device=DEV)
        keep = (rank < (case["top_k"] or vocab)).expand(n, -1)
        sw = torch.where(keep, sw, 0.0)
        run = sw.cumsum(1)
        if case["top_p"] < 1.0:
            goal = run[:, -1:] * float(torch.tensor(case["top_p"]))
            keep = keep & ((run - sw < goal) | (rank == 0))
        least = max(float(torch.tensor(case["min_p"])), 2.0 ** -FLOOR)
        w = torch.where(torch.zeros_like(keep).scatter(1, order, keep) & (w >= least), w, 0.0)
        run = w.cumsum(1)
        total = run[:, -1:]
        token = (run > s["uniform"].double()[:, None] * total).long().argmax(1)
        logprob = torch.log(w.gather(1, token[:, None]) / total)[:, 0].float()
    out = {"token": token.to(torch.int32), "logprob": logprob}
    if case["tree"]:
        out.update(_plain_walk(s["parent"], s["tokens"], out["token"]))
    return out


def _plain_walk(parent, tokens, target):
    n = parent.numel()
    node = torch.arange(n, device=DEV)
    up = parent.long().clamp(min=0)
    match = (tokens == target[up]) | (node == 0)
    # of several matching siblings the lowest index is followed
    rival = match[None, :] & (up[None, :] == up[:, None]) & (node[None, :] < node[:, None])
    match = match & (~(rival & (node > 0)[None, :]).any(1) | (node == 0))
    taken = (match[None, :] | ~_ancestors(parent)).all(1)
    length = taken.sum()
    path = torch.where(node < length, (~taken).int().sort(stable=True).indices, -1)
    nxt = path.roll(-1)
    emitted = torch.where(node + 1 < length, tokens[nxt.clamp(min=0)],
                          target[path.clamp(min=0)])
    return {"accept_len": length.to(torch.int32)[None], "path": path.to(torch.int32),
            "out_tokens": torch.where(node < length, emitted, -1).to(torch.int32)}


def _seen(s):
    """Which keys [rows, ctx] each of the last rows sees."""
    n, ctx, window = (s["case"][k] for k in ("rows", "ctx", "window"))
    at = torch.arange(ctx - n, ctx, device=DEV)[:, None]
    back = at - torch.arange(ctx, device=DEV)[None, :]
    return (back >= 0) & (back < (window or ctx + 1))


def _scores(s):
    """q . k / sqrt(d), [hkv, rows, group, ctx]."""
    case = s["case"]
    n, hq, hkv, d = (case[k] for k in ("rows", "hq", "hkv", "d"))
    g = hq // hkv
    q = s["q"].float().view(n, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, n * g, d)
    x = (q @ _values(s["k"], case).transpose(1, 2)) * (1.0 / math.sqrt(d))
    return x.view(hkv, n, g, -1)


def _plain_weigh(s):
    case = s["case"]
    n, hq, hkv, ctx = (case[k] for k in ("rows", "hq", "hkv", "ctx"))
    lse = s["lse"].view(n, hkv, hq // hkv).permute(1, 0, 2)[..., None]
    p = torch.exp(_scores(s) - lse)
    p = torch.where(_seen(s)[None, :, None, :], p, 0.0).sum((1, 2))
    had = torch.where(torch.arange(ctx, device=DEV) < ctx - n, s["weights"], 0.0)
    return {"weights": had + p}


def _plain_evict(s):
    case = s["case"]
    ctx, keep, sinks, recent = (case[k] for k in ("ctx", "keep", "sinks", "recent"))
    n = min(ctx, keep)
    at = torch.arange(ctx, device=DEV)
    bits = (s["weights"] + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 31) + (ctx - 1 - at)
    key = torch.where((at < sinks) | (at >= ctx - recent), (1 << 62) + (ctx - 1 - at), key)
    kept = key.topk(n, 1).indices.sort(1).values

    def rows(x):
        x = x.gather(1, kept[..., None].expand(-1, -1, x.shape[2]))
        x = _values(x, case)
        return x.to(torch.float16 if case["fmt"] == "f16" else torch.bfloat16)

    return {"kept": kept.to(torch.int32), "weights": s["weights"].gather(1, kept),
            "k": rows(s["k"]), "v": rows(s["v"])}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"encode": _plain_encode, "sample": _plain_sample, "weigh": _plain_weigh,
                "evict": _plain_evict}[op](s)
    from tree_verify_attention_gb300 import api
    if op == "encode":
        q, k, v = s["out"]
        if case["where"] == "given":
            place = {"positions": s["positions"]}
        else:
            place = {"ctx_len": s["ctx_len"], "dropped": s["dropped"], "parent": s.get("parent")}
        api.qk_norm_rope(s["q"], s["k"], s["v"], s["rope"], q, k, v, s["q_weight"],
                         s["k_weight"], eps=1e-6, **place)
        return {"q": q, "k": k, "v": v}
    if op == "sample":
        out = {"token": s["token"], "logprob": s["logprob"]}
        if not case["tree"]:
            api.sample_tokens(s["logits"], s["uniform"], s["sampling"], s["token"], s["logprob"])
            return out
        api.sample_accept(s["logits"], s["uniform"], s["sampling"], s["parent"], s["tokens"],
                          s["token"], s["accept_len"], s["path"], s["out_tokens"], s["ws"],
                          logprob=s["logprob"])
        return {**out, "accept_len": s["accept_len"], "path": s["path"],
                "out_tokens": s["out_tokens"]}
    if op == "weigh":
        api.kv_weights(s["cache"], s["q"], s["lse"], s["out"], prev=s["weights"],
                       window=case["window"])
        return {"weights": s["out"]}
    api.kv_evict(s["cache"], s["weights"], s["into"], s["kept"], sinks=case["sinks"],
                 recent=case["recent"], weights_out=s["weights_out"])
    out = {"kept": s["kept"], "weights": s["weights_out"]}
    if case["fmt"] == "f16":
        return {**out, "k": s["into"].k.view(torch.float16), "v": s["into"].v.view(torch.float16)}
    k, v = s["rows_out"]
    s["into"].read(0, k.shape[1], k, v, head_major=True)
    return {**out, "k": k, "v": v}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The operators from their definitions in 64 bits, on run()'s inputs."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"encode": _exact_encode, "sample": _exact_sample, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](s)


def _exact_encode(s):
    case = s["case"]
    n, rot = case["rows"], case["rot"]
    if case["where"] == "given":
        pos = s["positions"].tolist()
    else:
        base = int(s["ctx_len"]) + int(s["dropped"])
        deep = list(range(n))
        if case["where"] == "tree":
            for i, p in enumerate(s["parent"].tolist()):
                deep[i] = 0 if i == 0 else deep[p] + 1
        pos = [base + i for i in deep]
    pos = torch.tensor(pos, dtype=torch.float64, device=DEV)
    turn = torch.ones(n, rot // 2, dtype=torch.complex128, device=DEV)
    for i in range(rot // 2):
        a = pos * math.pow(1e6, -2.0 * i / rot)
        turn[:, i] = torch.complex(torch.cos(a), torch.sin(a))
    out = {"v": s["v"].double()}
    for name in ("q", "k"):
        x = s[name].double()
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6)
        x = x * s[name + "_weight"].double()
        one, two = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["pairs"] == "half"
                    else (slice(0, rot, 2), slice(1, rot, 2)))
        c = torch.complex(x[..., one], x[..., two]) * turn[:, None]
        x[..., one], x[..., two] = c.real, c.imag
        out[name] = x
    return out


def _exact_sample(s):
    case = s["case"]
    n, vocab = s["logits"].shape
    logprob = torch.zeros(n, dtype=torch.float64, device=DEV)
    none = {"token": None, "logprob": logprob}
    if case["tree"]:
        none.update({"accept_len": None, "path": None, "out_tokens": None})
    if case["temperature"] == 0.0:
        return none
    p_goal = float(torch.tensor(case["top_p"], dtype=torch.float32))
    p_min = float(torch.tensor(case["min_p"], dtype=torch.float32))
    t = float(torch.tensor(case["temperature"], dtype=torch.float32))
    for r in range(n):
        x, who = torch.sort(s["logits"][r].double(), descending=True, stable=True)
        p = torch.softmax(x / t, 0)
        last = case["top_k"] if 0 < case["top_k"] < vocab else vocab
        p, who = p[:last] / p[:last].sum(), who[:last]
        if p_goal < 1.0:
            below = torch.cat((p.new_zeros(1), p.cumsum(0)[:-1]))
            last = max(1, int((below < p_goal).sum()))
            p, who = p[:last], who[:last]
        last = int((p >= p[0] * max(p_min, 2.0 ** -FLOOR)).sum())
        p, who = p[:last], who[:last]
        back = torch.argsort(who)
        p = p[back]
        run = p.cumsum(0)
        at = torch.searchsorted(run, s["uniform"][r].double() * run[-1], right=True)
        logprob[r] = torch.log(p[at.clamp(max=last - 1)] / run[-1])
    return none


def _exact_weigh(s):
    case = s["case"]
    n, hq, hkv, d, ctx, window = (case[k] for k in ("rows", "hq", "hkv", "d", "ctx", "window"))
    out = s["weights"].double()
    out[:, ctx - n:] = 0.0
    for h in range(hkv):
        k = _values(s["k"][h], case, torch.float64)
        for i in range(n):
            last = ctx - n + i
            first = 0 if window == 0 else max(0, last - window + 1)
            q = s["q"][i, h * (hq // hkv):(h + 1) * (hq // hkv)].double()
            lse = s["lse"][i, h * (hq // hkv):(h + 1) * (hq // hkv)].double()
            x = torch.einsum("gd,td->gt", q, k[first:last + 1]) / math.sqrt(d)
            out[h, first:last + 1] += torch.exp(x - lse[:, None]).sum(0)
    return {"weights": out}


def _exact_evict(s):
    case = s["case"]
    ctx, sinks, recent = case["ctx"], case["sinks"], case["recent"]
    n = min(ctx, case["keep"])
    out = {"kept": None, "weights": [], "k": [], "v": []}
    for h in range(case["hkv"]):
        w = s["weights"][h].double()
        w[:sinks] = math.inf
        w[ctx - recent:] = math.inf
        kept = torch.sort(w, descending=True, stable=True).indices[:n].sort().values
        out["weights"].append(s["weights"][h][kept].double())
        for name in ("k", "v"):
            out[name].append(_values(s[name][h][kept], case, torch.float64))
    return {k: v if v is None else torch.stack(v) for k, v in out.items()}
