"""Cases, plain forms and calls of the operators around the 8-bit KV cache.

Four operators, each over the sizes a verify loop and the server around it
meet:

* ``write``  -- K and V rows quantised to 8 bits as they enter the cache (one
  scale for each block of 64 positions and head; the open block stays bf16),
  and the touched rows read back as the values they now stand for;
* ``read``   -- rows of the cache read back;
* ``attend`` -- attention of the draft-tree nodes (one node: plain decode)
  over the committed 8-bit cache and their own ancestors;
* ``score``  -- log probabilities of given tokens, the entropy of each row of
  logits and its top alternatives.

``own = False`` runs the plain forms (elementary torch operations, 32 bits,
rounded once at the end); ``own = True`` makes the calls a user makes.
"""

import math

import torch

own = False

BLOCK = 64           # positions that share a scale
DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a few accepted rows (budget 22) entering a long cache, ending inside a block
        {"name": "write_accepted", "op": "write", "rows": 9, "at": 61477, "hkv": 4, "d": 256,
         "src": "bf16"},
        # a prompt of odd length, from float32 rows, eight heads of 128, behind a short prefix
        {"name": "write_prompt_f32", "op": "write", "rows": 4001, "at": 100, "hkv": 8, "d": 128,
         "src": "f32"},
        # the long-context prompt (ctx 61440, four heads of 256)
        {"name": "write_prompt_long", "op": "write", "rows": 61440, "at": 0, "hkv": 4, "d": 256,
         "src": "bf16"},
        # a tiny cache (ctx 256, one head of 64) read back as float32, odd bounds
        {"name": "read_tiny", "op": "read", "ctx": 256, "pos": 3, "rows": 251, "hkv": 1, "d": 64,
         "dst": "f32"},
        # a 32768-row cache handed to a bf16 consumer
        {"name": "read_32768", "op": "read", "ctx": 32768, "pos": 0, "rows": 32768, "hkv": 4,
         "d": 256, "dst": "bf16"},
        # autoregressive decode: one token over a 128K context
        {"name": "attend_decode_128k", "op": "attend", "nodes": 1, "hq": 24, "hkv": 4, "d": 256,
         "ctx": 131060, "window": 0},
        # the verify step's attention: budget 22, 2048-token window, ctx 61440
        {"name": "attend_tree_window", "op": "attend", "nodes": 23, "hq": 24, "hkv": 4, "d": 256,
         "ctx": 61440, "window": 2048},
        # the same tree over the whole 128K context
        {"name": "attend_tree_128k", "op": "attend", "nodes": 23, "hq": 24, "hkv": 4, "d": 256,
         "ctx": 131072, "window": 0},
        # the largest budget, heads of 128, an odd context
        {"name": "attend_tree64_odd", "op": "attend", "nodes": 65, "hq": 32, "hkv": 8, "d": 128,
         "ctx": 32791, "window": 0},
        # one sampled token's log probability with twenty alternatives
        {"name": "score_token", "op": "score", "rows": 1, "vocab": 151936, "top": 20,
         "src": "f32", "banned": 0},
        # every node of a verify step
        {"name": "score_tree", "op": "score", "rows": 23, "vocab": 151936, "top": 8,
         "src": "bf16", "banned": 500},
        # the tokens of a prompt scored
        {"name": "score_prompt", "op": "score", "rows": 1024, "vocab": 151936, "top": 5,
         "src": "bf16", "banned": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "score"])
    if op == "score":
        vocab = _log_int(rng, 33, 151936)
        rows = _log_int(rng, 1, max(1, min(4096, 1024 * 151936 // vocab)))
        return {"op": op, "rows": rows, "vocab": vocab, "top": rng.randint(0, 32),
                "src": rng.choice(["bf16", "f32"]) if rows * vocab < 4e7 else "bf16",
                "banned": rng.choice([0, 0, rng.randint(1, vocab - 1)])}
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "write":
        most = 61440 * 4 * 256 // (hkv * d)
        rows = _log_int(rng, 1, min(131072, most))
        return {"op": op, "rows": rows, "at": rng.choice([0, rng.randint(0, 4096)]), "hkv": hkv,
                "d": d, "src": rng.choice(["bf16", "f32"]) if 2 * rows < most else "bf16"}
    if op == "read":
        ctx = _log_int(rng, 1, min(131072, 32768 * 4 * 256 // (hkv * d)))
        rows = _log_int(rng, 1, ctx)
        return {"op": op, "ctx": ctx, "pos": rng.randint(0, ctx - rows), "rows": rows,
                "hkv": hkv, "d": d, "dst": rng.choice(["bf16", "f32"]) if 2 * rows <= ctx else "bf16"}
    group = rng.choice([1, 2, 4, 5, 6, 8])
    nodes = rng.choice([1, 1, rng.randint(2, 65)])
    most = 131072 * 4 * 256 // (hkv * d)
    most = min(131072, most, int(131072 * 24 * 23 * 256 / (hkv * group * d * nodes)))
    ctx = _log_int(rng, 1, most)
    return {"op": op, "nodes": nodes, "hq": hkv * group, "hkv": hkv, "d": d, "ctx": ctx,
            "window": rng.choice([0, 0, _log_int(rng, 1, 4096)])}


def work(case):
    op = case["op"]
    if op == "score":
        n, v, k = case["rows"], case["vocab"], case["top"]
        size = 4 if case["src"] == "f32" else 2
        return {"bytes": n * v * size + n * (4 + 4 + 4 + 8 * k), "flops": 6.0 * n * v}
    hkv, d = case["hkv"], case["d"]
    if op == "write":
        first = case["at"] // BLOCK * BLOCK
        n, back = case["rows"], case["at"] + case["rows"] - first
        size = 4 if case["src"] == "f32" else 2
        # rows in, codes out, and the values read back
        return {"bytes": 2 * hkv * d * (n * (size + 1) + back * 2), "flops": 2.0 * hkv * d * n * 4}
    if op == "read":
        size = 4 if case["dst"] == "f32" else 2
        return {"bytes": 2 * hkv * d * case["rows"] * (1 + size),
                "flops": 2.0 * hkv * d * case["rows"]}
    n, hq, ctx = case["nodes"], case["hq"], case["ctx"]
    seen = ctx if case["window"] == 0 else min(ctx, case["window"] - 1)
    tail = min(ctx % BLOCK, seen)
    moved = 2 * hkv * ((seen - tail) * (d + 4 / BLOCK) + (tail + n) * d * 2)
    return {"bytes": moved + n * hq * (d * 4 + 4) + 4 * n,
            "flops": 4.0 * d * hq * n * (seen + 1)}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(g, n, hkv, d, dtype):
    """K or V rows [n, hkv, d]: unit normals, some channels a few times larger."""
    x = torch.randn(n, hkv, d, generator=g, device=DEV)
    x = x * (1.0 + 3.0 * (torch.rand(hkv, d, generator=g, device=DEV) < 0.03).float())
    return x.to(dtype)


def _cached(g, n_blocks, hkv, d):
    """A filled cache in the layout the library documents: per 64-position
    block and head, 8-bit codes and one scale; K codes as [d / 16][64][16]
    bytes, V codes as [4][d][16] bytes (16 positions innermost)."""
    out = []
    for is_v in (False, True):
        codes = torch.empty(hkv, n_blocks, BLOCK * d, dtype=torch.int8, device=DEV)
        scale = torch.empty(hkv, n_blocks, device=DEV)
        for h in range(hkv):
            x = _rows(g, n_blocks * BLOCK, 1, d, torch.bfloat16).float().view(n_blocks, BLOCK, d)
            amax = x.abs().amax((1, 2))
            c = (x * 127.0 / amax[:, None, None]).round().to(torch.int8)
            c = (c.view(n_blocks, 4, 16, d).transpose(2, 3) if is_v
                 else c.view(n_blocks, BLOCK, d // 16, 16).transpose(1, 2))
            codes[h] = c.reshape(n_blocks, BLOCK * d)
            scale[h] = amax / 127.0
        shape = (hkv, n_blocks, 4, d, 16) if is_v else (hkv, n_blocks, d // 16, BLOCK, 16)
        tail = _rows(g, 2 * BLOCK, hkv, d, torch.bfloat16).view(2, BLOCK, hkv, d)
        out.append((codes.view(shape), scale, tail.permute(2, 0, 1, 3).contiguous()))
    return out


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
    return torch.tensor(parent, dtype=torch.int32)


def _floats(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "score":
        n, v = case["rows"], case["vocab"]
        x = torch.randn(n, v, generator=g, device=DEV) * 2.5
        hit = torch.randint(0, v, (n,), generator=g, device=DEV)
        x[torch.arange(n, device=DEV), hit] += 12.0       # a model that is often sure
        if case["banned"]:
            first = int(torch.randint(0, v - case["banned"] + 1, (1,), generator=g, device=DEV))
            x[:, first:first + case["banned"]] = -math.inf
        s["logits"] = x.to(_floats(case["src"]))
        other = torch.randint(0, v, (n,), generator=g, device=DEV)
        pick = torch.rand(n, generator=g, device=DEV) < 0.7
        s["tokens"] = torch.where(pick, hit, other).to(torch.int32)
        if own:
            s["out"] = (torch.empty(n, device=DEV), torch.empty(n, device=DEV),
                        torch.empty(n, case["top"], dtype=torch.int32, device=DEV),
                        torch.empty(n, case["top"], device=DEV))
        return s
    hkv, d = case["hkv"], case["d"]
    ctx = case["at"] if op == "write" else case["ctx"]
    extra = case["rows"] if op == "write" else case.get("nodes", 0)
    blocks = -(-(ctx + extra) // BLOCK)
    if op == "write":
        # the rows of the open block are all that a write reads of the cache
        s["k_tail"], s["v_tail"] = (
            _rows(g, 2 * BLOCK, hkv, d, torch.bfloat16).view(2, BLOCK, hkv, d)
            .permute(2, 0, 1, 3).contiguous() for _ in range(2))
        s["k_rows"] = _rows(g, case["rows"], hkv, d, _floats(case["src"]))
        s["v_rows"] = _rows(g, case["rows"], hkv, d, _floats(case["src"]))
    else:
        (s["k"], s["k_scale"], s["k_tail"]), (s["v"], s["v_scale"], s["v_tail"]) = _cached(
            g, blocks, hkv, d)
    if op == "attend":
        n, hq = case["nodes"], case["hq"]
        s["q"] = torch.randn(n, hq, d, generator=g, device=DEV).to(torch.bfloat16)
        s["tree_k"] = _rows(g, n, hkv, d, torch.bfloat16)
        s["tree_v"] = _rows(g, n, hkv, d, torch.bfloat16)
        s["parent"] = _tree(seed, n).to(DEV)
    if own:
        from tree_verify_attention_gb300 import api
        cache = api.Int8Cache(hkv, d, ctx + extra, device=DEV)
        for name in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail"):
            if name in s:
                getattr(cache, name).copy_(s.pop(name))
        cache.ctx_len.fill_(ctx)
        s["cache"] = cache
        if op == "attend":
            s["out"] = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
            s["lse"] = torch.empty(n, hq, device=DEV)
            s["ws"] = api.workspace(api.int8_attn_workspace_bytes(
                n, hq, hkv, d, case["window"], cache.capacity), device=DEV)
        else:
            n = case["rows"] if op == "read" else ctx + extra - ctx // BLOCK * BLOCK
            dtype = _floats(case.get("dst"))
            s["out"] = tuple(torch.empty(n, hkv, d, dtype=dtype, device=DEV) for _ in range(2))
    return s


# ---------------------------------------------------------------- plain forms

def _plain_write(s):
    """K and V rows from the start of the open block on, as the cache holds
    them after the write: whole blocks rounded to 8 bits, the open one bf16."""
    case = s["case"]
    at, n, hkv, d = case["at"], case["rows"], case["hkv"], case["d"]
    first = at // BLOCK
    kept = at - first * BLOCK
    total = kept + n
    whole = total // BLOCK * BLOCK

    def one(tail, rows):
        old = tail[:, first % 2, :kept].transpose(0, 1)
        x = torch.cat([old, rows.to(torch.bfloat16)]).float()
        b = x[:whole].reshape(-1, BLOCK, hkv, d)
        amax = b.abs().amax((1, 3), keepdim=True)
        code = (b * 127.0 / amax).round()
        back = (code * (amax / 127.0)).reshape(whole, hkv, d)
        return torch.cat([back, x[whole:]]).to(torch.bfloat16)

    return {"k": one(s["k_tail"], s["k_rows"]), "v": one(s["v_tail"], s["v_rows"])}


def _plain_rows(s, pos, end):
    """Cached K and V at positions [pos, end) as float32 [hkv, end - pos, d]."""
    case = s["case"]
    hkv, d, ctx = case["hkv"], case["d"], case["ctx"]
    b0, closed = pos // BLOCK, ctx // BLOCK
    b1 = min(-(-end // BLOCK), closed)

    def one(codes, scale, tail, is_v):
        c = codes[:, b0:b1]
        c = c.transpose(3, 4) if is_v else c.transpose(2, 3)     # positions before dims
        x = c.reshape(hkv, (b1 - b0), BLOCK, d).float() * scale[:, b0:b1, None, None]
        x = x.reshape(hkv, (b1 - b0) * BLOCK, d)
        x = torch.cat([x, tail[:, closed % 2, :ctx - closed * BLOCK].float()], 1)
        return x[:, pos - b0 * BLOCK:end - b0 * BLOCK]

    return (one(s["k"], s["k_scale"], s["k_tail"], False),
            one(s["v"], s["v_scale"], s["v_tail"], True))


def _plain_read(s):
    case = s["case"]
    k, v = _plain_rows(s, case["pos"], case["pos"] + case["rows"])
    dtype = _floats(case["dst"])
    return {"k": k.transpose(0, 1).to(dtype), "v": v.transpose(0, 1).to(dtype)}


def _ancestors(parent):
    """Ancestor-or-self matrix [n, n] of a tree, from powers of its adjacency."""
    n = parent.numel()
    step = torch.eye(n, dtype=torch.float64, device=parent.device)
    step[torch.arange(1, n, device=parent.device), parent[1:].long()] = 1.0
    return torch.linalg.matrix_power(step, 64) > 0


def _plain_attend(s):
    case = s["case"]
    n, hq, hkv, d, ctx, window = (case[k] for k in ("nodes", "hq", "hkv", "d", "ctx", "window"))
    lo = 0 if window == 0 else max(0, ctx - window + 1)
    if lo < ctx:
        k, v = _plain_rows(s, lo, ctx)
    else:
        k = v = torch.empty(hkv, 0, d, device=DEV)
    k = torch.cat([k, s["tree_k"].float().transpose(0, 1)], 1)
    v = torch.cat([v, s["tree_v"].float().transpose(0, 1)], 1)
    anc = _ancestors(s["parent"])
    depth = anc.sum(1) - 1
    pos = torch.arange(lo, ctx, device=DEV)
    near = (ctx + depth[:, None] - pos[None, :] < window) if window else (pos >= 0).expand(n, -1)
    seen = torch.cat([near, anc], 1)
    g = hq // hkv
    q = s["q"].float().view(n, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, n * g, d)
    x = (q @ k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    x = x.view(hkv, n, g, -1).masked_fill(~seen[None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (p.view(hkv, n * g, -1) @ v).view(hkv, n, g, d) / total
    lse = (m + torch.log(total))[..., 0]
    return {"out": o.permute(1, 0, 2, 3).reshape(n, hq, d).to(torch.bfloat16),
            "lse": lse.permute(1, 0, 2).reshape(n, hq)}


def _plain_score(s):
    x, top = s["logits"].float(), s["case"]["top"]
    n, vocab = x.shape
    m = x.amax(1, keepdim=True)
    z = x - m
    e = torch.exp(z)
    total = e.sum(1)
    lse = m[:, 0] + torch.log(total)
    entropy = torch.log(total) - torch.where(e > 0, e * z, 0.0).sum(1) / total
    logprob = x.gather(1, s["tokens"].long()[:, None])[:, 0] - lse
    # one whole number for each value that orders by value, then by lower index
    bits = (x + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32)
    key = key + (vocab - 1 - torch.arange(vocab, device=x.device))
    ids = vocab - 1 - (key.topk(top, 1).values & 0xFFFFFFFF)
    return {"logprob": logprob, "entropy": entropy, "top_ids": ids.to(torch.int32),
            "top_logprobs": x.gather(1, ids) - lse[:, None]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend,
                "score": _plain_score}[op](s)
    from tree_verify_attention_gb300 import api
    if op == "write":
        s["cache"].append(s["k_rows"], s["v_rows"], at=s["case"]["at"])
        k, v = s["out"]
        s["cache"].read(s["case"]["at"] // BLOCK * BLOCK, k.shape[0], k, v)
        return {"k": k, "v": v}
    if op == "read":
        k, v = s["out"]
        s["cache"].read(s["case"]["pos"], s["case"]["rows"], k, v)
        return {"k": k, "v": v}
    if op == "attend":
        api.tree_verify_attn(s["cache"], s["q"], s["tree_k"], s["tree_v"], s["parent"],
                             s["case"]["window"], 65, s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    logprob, entropy, top_ids, top_logprobs = s["out"]
    api.token_logprobs(s["logits"], s["tokens"], logprob, entropy, top_ids, top_logprobs)
    return {"logprob": logprob, "entropy": entropy, "top_ids": top_ids,
            "top_logprobs": top_logprobs}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The operators from their definitions in 64 bits, on run()'s inputs."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "score":
        return _exact_score(s)
    hkv, d = case["hkv"], case["d"]
    if op == "write":
        at, n = case["at"], case["rows"]
        start = at // BLOCK * BLOCK
        out = {}
        for name in ("k", "v"):
            tail, rows = s[name + "_tail"], s[name + "_rows"].to(torch.bfloat16)
            slot = (start // BLOCK) % 2
            res = torch.empty(at + n - start, hkv, d, dtype=torch.float64, device=DEV)
            for h in range(hkv):
                x = torch.cat((tail[h, slot, :at - start], rows[:, h])).double()
                full = len(x) // BLOCK
                cut = x[:full * BLOCK].reshape(full, BLOCK * d)
                unit = cut.abs().max(1, keepdim=True).values / 127 if full else cut[:, :1]
                res[:full * BLOCK, h] = (torch.round(cut / unit) * unit).reshape(-1, d)
                res[full * BLOCK:, h] = x[full * BLOCK:]
            out[name] = res
        return out
    ctx = case["ctx"]
    done = ctx // BLOCK

    def decode(h, lo, hi):
        """K and V of head h at positions [lo, hi)."""
        p = torch.arange(lo, hi, device=DEV)
        b, t = torch.div(p, BLOCK, rounding_mode="floor"), p % BLOCK
        held = b < done
        bb = b.clamp(max=max(done - 1, 0))
        rows = []
        for name in ("k", "v"):
            c = s[name][h]
            if name == "k":      # [blocks][d / 16][64][16]
                row = c[bb, :, t, :].reshape(len(p), d)
            else:                # [blocks][4][d][16]
                row = c[bb, torch.div(t, 16, rounding_mode="floor"), :, t % 16]
            val = row.double() * s[name + "_scale"][h][bb].double()[:, None]
            val[~held] = s[name + "_tail"][h, done % 2][t[~held]].double()
            rows.append(val)
        return rows

    if op == "read":
        pos, n = case["pos"], case["rows"]
        both = [decode(h, pos, pos + n) for h in range(hkv)]
        return {"k": torch.stack([b[0] for b in both], 1),
                "v": torch.stack([b[1] for b in both], 1)}
    n, hq, window = case["nodes"], case["hq"], case["window"]
    parent = s["parent"].tolist()
    line = []                    # each node's ancestors and itself
    for i in range(n):
        line.append(([] if i == 0 else line[parent[i]]) + [i])
    allowed = torch.zeros(n, n, dtype=torch.bool)
    for i, who in enumerate(line):
        allowed[i, who] = True
    allowed = allowed.to(DEV)
    lo = 0 if window == 0 else max(0, ctx - window + 1)
    out = torch.empty(n, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(n, hq, dtype=torch.float64, device=DEV)
    first = torch.tensor([0 if window == 0 else max(0, ctx + len(w) - window) for w in line],
                         device=DEV)
    old = torch.arange(lo, ctx, device=DEV)[None, :] >= first[:, None]
    mask = torch.cat((old, allowed), 1)
    for h in range(hkv):
        k, v = decode(h, lo, ctx)
        k = torch.cat((k, s["tree_k"][:, h].double()))
        v = torch.cat((v, s["tree_v"][:, h].double()))
        for r in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
            w = (s["q"][:, r].double() @ k.T) / math.sqrt(d)
            w[~mask] = -math.inf
            lse[:, r] = torch.logsumexp(w, 1)
            out[:, r] = torch.exp(w - lse[:, r:r + 1]) @ v
    return {"out": out, "lse": lse}


def _exact_score(s):
    n, top = s["case"]["rows"], s["case"]["top"]
    parts = []
    for r in range(0, n, 64):
        x = s["logits"][r:r + 64].double()
        logp = torch.log_softmax(x, 1)
        held = torch.where(torch.isinf(logp), 0.0, logp)
        parts.append((logp.gather(1, s["tokens"][r:r + 64].long()[:, None])[:, 0],
                      -(torch.exp(logp) * held).sum(1),
                      logp.topk(top, 1).values))
    lp, entropy, best = (torch.cat(c) for c in zip(*parts))
    return {"logprob": lp, "entropy": entropy, "top_ids": None, "top_logprobs": best}
