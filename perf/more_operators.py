"""Measured cases of the verification of drafted token trees and of sampling from logits: their
inputs, their plain forms in elementary torch operations, the framework's calls, and their
definitions in 64 bits.

A request's packed rows cu[r] .. cu[r + 1] - 1 are the nodes of its tree: row 0 is the anchor, every
other row a drafted token with a parent before it in the segment.  A node sees the request's
committed tokens, itself and its ancestors.  Three passes of such a step:

* ``attn``: the attention of the packed nodes over the paged cache;
* ``sample``: one token a row from filtered, tempered logits, given exponential noise, and where
  asked for the distribution that it comes from;
* ``tree``: what a step does around its forward pass: visibility masks and positions from the
  parents, then the walk down the tree along the sampled tokens and the commit of its rows.
"""
import math

import torch

own = False

D = 128       # head dim
GAMMA = 16    # most drafted tokens that a step commits


# ---------------------------------------------------------------- cases
def _attn(name, b, n_lo, n_hi, c_lo, c_hi, hq, hkv, page):
    return {"name": name, "op": "attn", "b": b, "n_lo": n_lo, "n_hi": n_hi, "c_lo": c_lo,
            "c_hi": c_hi, "hq": hq, "hkv": hkv, "page": page}


def _sample(name, b, per, vocab, dtype, probs, params, pad):
    """b requests of `per` rows each; probs: the distribution's type or "none"; params: the kind of
    the requests' parameters; pad: elements between the rows of the logits."""
    return {"name": name, "op": "sample", "b": b, "per": per, "vocab": vocab, "dtype": dtype,
            "probs": probs, "params": params, "pad": pad}


def _tree(name, b, n_lo, n_hi, c_hi, hkv, page):
    return {"name": name, "op": "tree", "b": b, "n_lo": n_lo, "n_hi": n_hi, "c_lo": 1, "c_hi": c_hi,
            "hkv": hkv, "page": page}


def listed():
    return [
        # a small tree of one request, a short context: latency alone
        _attn("attn_tree_one", 1, 9, 9, 997, 997, 32, 8, 16),
        # many requests that verify single tokens, as when nothing was drafted
        _attn("attn_tree_single", 256, 1, 1, 512, 4096, 40, 8, 16),
        # a serving batch: ragged trees over ragged contexts
        _attn("attn_tree_batch", 32, 17, 64, 1024, 4096, 32, 8, 16),
        # large trees, several row tiles to a request
        _attn("attn_tree_large", 16, 97, 256, 2048, 8192, 40, 8, 64),
        # few requests with long contexts
        _attn("attn_tree_long", 2, 26, 33, 131071, 131071, 40, 8, 64),
        # one row of one request: latency alone
        _sample("sample_one", 1, 1, 151936, "f32", "none", "mixed", 0),
        # the rows of a verification step with their distributions, every kind of request among them
        _sample("sample_verify", 32, 9, 151936, "f32", "f32", "mixed", 0),
        # many requests' single rows in bf16, tokens alone, top-p throughout
        _sample("sample_top_p", 256, 4, 129280, "bf16", "none", "top_p", 0),
        # an odd vocabulary whose rows do not lie densely
        _sample("sample_odd", 67, 5, 50257, "bf16", "bf16", "mixed", 3),
        # one request's tree
        _tree("tree_one", 1, 9, 9, 500, 8, 16),
        # a serving batch
        _tree("tree_batch", 32, 17, 64, 400, 8, 16),
        # the largest batch, a few requests without a node
        _tree("tree_wide", 256, 0, 64, 300, 8, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("attn", "attn", "sample", "sample", "tree"))
    hq, hkv = rng.choice(((8, 2), (20, 4), (32, 8), (40, 8), (32, 4), (16, 16), (7, 1)))
    page = rng.choice((16, 16, 32, 64, 128))
    if op == "attn":
        n = rng.choice((1, _log(rng, 2, 17), _log(rng, 16, 64), _log(rng, 17, 256)))
        b = _log(rng, 1, max(1, min(256, 2500 // n)))
        # no more keys and no more products than the largest listed cases
        hi = _log(rng, 1, min(120000, 260000 // b, 30000000 // (b * n)))
        c = _attn("", b, rng.randint((n + 1) // 2, n), n, rng.randint(hi // 3, hi), hi, hq, hkv, page)
    elif op == "sample":
        v = _log(rng, 100, 152000)
        b = _log(rng, 1, max(1, min(256, 60000000 // v)))
        per = rng.randint(1, max(1, min(17, 60000000 // (v * b))))
        c = _sample("", b, per, v, rng.choice(("f32", "bf16")), rng.choice(("none", "f32", "bf16")),
                    rng.choice(("mixed", "mixed", "top_p", "top_k", "off")), rng.choice((0, 0, 3, 64)))
    else:
        n = _log(rng, 1, 64)
        c = _tree("", _log(rng, 1, 256), rng.randint(n // 2, n), n, _log(rng, 2, 280), hkv, page)
    del c["name"]
    return c


def _spread(lo, hi, b):
    """b lengths over [lo, hi], the same for every seed: a case's work is its own."""
    return [lo + (i * 7919 + 13) % (hi - lo + 1) for i in range(b)]


def _params(c):
    """(temperature, top_k, top_p, min_p) of a case's requests: greedy, plain and filtered ones."""
    t, k, p, m = [], [], [], []
    for i in range(c["b"]):
        kind = i % 7 if c["params"] == "mixed" else -1
        t.append(0.0 if kind == 4 else 0.6 + 0.1 * (i % 6))
        k.append(50 if kind in (0, 1) else 1000 if kind == 5 else 0)
        p.append(0.95 if kind in (0, 5) else 0.9 if kind == 2 else 1.0)
        m.append(0.05 if kind in (1, 6) else 0.0)
        if c["params"] == "top_p":
            p[-1] = 0.8 + 0.03 * (i % 6)
        if c["params"] == "top_k":
            k[-1] = 1 + (i * 37) % 300
    return t, k, p, m


def work(case):
    c = case
    if c["op"] == "attn":
        n, p = _spread(c["n_lo"], c["n_hi"], c["b"]), _spread(c["c_lo"], c["c_hi"], c["b"])
        rows, products = sum(n), sum(a * b for a, b in zip(n, p))
        # a node has some ancestors: the products inside the blocks are left out
        by = (sum(p) * c["hkv"] * 2 + rows * (2 * c["hq"] + 2 * c["hkv"])) * D * 2.0
        return {"bytes": by + rows * (4.0 * c["hq"] + 8 * ((c["n_hi"] + 63) // 64)),
                "flops": 4.0 * products * c["hq"] * D}
    if c["op"] == "sample":
        rows, size = c["b"] * c["per"], {"f32": 4, "bf16": 2, "none": 0}
        noise = 0  # of the tokens that no filter takes out for sure
        for t, k, p, m in zip(*_params(c)):
            if t > 0:
                noise += min(k, c["vocab"]) if k else (c["vocab"] if p >= 1 and m <= 0 else 0)
        return {"bytes": rows * c["vocab"] * float(size[c["dtype"]] + size[c["probs"]]) +
                noise * c["per"] * 4.0, "flops": 8.0 * rows * c["vocab"]}
    n = _spread(c["n_lo"], c["n_hi"], c["b"])
    # parents, tokens and samples in, masks and positions out; some rows a request moved
    return {"bytes": sum(n) * 24.0 + c["b"] * 3 * c["hkv"] * D * 8.0, "flops": sum(n) * 8.0}


# ---------------------------------------------------------------- inputs
def _pages(tokens, spare, page, gen, dev):
    """A table of distinct pages in random order for requests of these token counts, `spare` columns
    wider than the longest, and the pages that are left."""
    need = [(t + page - 1) // page for t in tokens]
    n_pages = sum(need) + spare * len(tokens) + 3
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    width = max(max(need), 1) + spare
    col = torch.arange(width, device=dev)
    cnt = torch.tensor(need, device=dev)
    first = torch.cumsum(cnt, 0) - cnt
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    table = torch.where(col < cnt[:, None], perm[at], torch.zeros_like(perm[at]))
    return table, n_pages, perm[sum(need):].contiguous()


def _forest(c, gen, dev):
    """Row counts, first rows, the request and the index in its segment of every row, and the rows'
    parents: a node hangs off one of the four rows before it or off any, so that depths of a dozen
    and wide levels both occur."""
    n = _spread(c["n_lo"], c["n_hi"], c["b"])
    cu = torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)
    rows = max(sum(n), 1)
    req = torch.repeat_interleave(torch.arange(c["b"], device=dev), torch.tensor(n, device=dev))
    i = torch.arange(sum(n), device=dev) - cu[req]
    u = torch.rand(2, sum(n), generator=gen, device=dev)
    near = i - 1 - torch.minimum((u[1] * 4).long(), i - 1)
    parent = torch.where(u[0] < 0.5, near, (u[1] * i).long().clamp(max=i - 1)).to(torch.int32)
    parent[i == 0] = -1
    full = torch.full((rows,), -1, dtype=torch.int32, device=dev)
    full[:sum(n)] = parent
    return n, cu, rows, req, i, full


def _ancestors(parent, cu, req, i, width):
    """bool [rows, width]: row sees the block row of that index (itself or an ancestor)."""
    rows = req.numel()
    sees = torch.arange(width, device=i.device) == i[:, None]
    up, base = parent[:rows].long(), cu[req].long()
    at = torch.where(up >= 0, base + up, torch.full_like(up, -1))
    for _ in range(width.bit_length()):     # up: 1, 2, 4, ... generations
        sees = sees | torch.where((at >= 0)[:, None], sees[at.clamp(min=0)], torch.zeros_like(sees))
        at = torch.where(at >= 0, at[at.clamp(min=0)], at)
    return sees


def _words(sees):
    """bool [rows, 64 w] -> int64 [rows, w], bit j of word w the column 64 w + j."""
    bit = torch.ones(64, dtype=torch.int64, device=sees.device) << torch.arange(64, device=sees.device)
    return (sees.unflatten(1, (-1, 64)).to(torch.int64) * bit).sum(-1)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 29)
    if c["op"] == "sample":
        return _prepare_sample(c, gen, dev)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=dev).to(torch.bfloat16)

    n, cu, rows, req, i, parent = _forest(c, gen, dev)
    ctx = _spread(c["c_lo"], c["c_hi"], c["b"])
    hkv, page = c["hkv"], c["page"]
    words = (max(max(n), 1) + 63) // 64
    state = {"case": c, "cu": cu, "req": req, "i": i, "rows": rows, "parent": parent,
             "ctx": torch.tensor(ctx, dtype=torch.int32, device=dev), "words": words,
             "width": max(max(n), 1), "length": max(ctx)}
    spare = 0 if c["op"] == "attn" else 2 + GAMMA // page
    table, n_pages, left = _pages(ctx, spare, page, gen, dev)
    state.update(table=table, k_cache=rand(n_pages, page, hkv, D), v_cache=rand(n_pages, page, hkv, D),
                 k_new=rand(rows, hkv, D), v_new=rand(rows, hkv, D))
    if c["op"] == "attn":
        hq = c["hq"]
        mask = torch.zeros(rows, words, dtype=torch.int64, device=dev)
        mask[:req.numel()] = _words(_ancestors(parent, cu, req, i, 64 * words))
        state.update(q=1.5 * rand(rows, hq, D), mask=mask, scale=1.0 / math.sqrt(D),
                     out=torch.zeros(rows, hq, D, dtype=torch.bfloat16, device=dev),
                     lse=torch.zeros(rows, hq, dtype=torch.float32, device=dev))
        if own:  # the workspace that a serving program keeps for its steps
            import speculative_decoding_verification_dspark_gb300 as dspark
            state["ws"] = torch.empty(dspark.verify_attn_tree_workspace_size(
                c["b"], rows, hq, hkv, 32, max(n)), dtype=torch.uint8, device=dev)
        return state
    # drafted tokens, and samples that often are the token of one of the row's children
    b, live = c["b"], req.numel()

    def empty(*shape, dtype=torch.int32):
        return torch.zeros(*shape, dtype=dtype, device=dev)

    tok = torch.randint(0, 151936, (rows,), generator=gen, device=dev, dtype=torch.int32)
    picked = torch.randint(0, 151936, (rows,), generator=gen, device=dev, dtype=torch.int32)
    follow = torch.rand(live, generator=gen, device=dev) < 0.6
    at = (cu[req] + parent[:live]).long()
    hit = (parent[:live] >= 0) & follow
    child = torch.full((rows,), -1, device=dev).scatter_reduce_(
        0, at[hit], torch.arange(live, device=dev)[hit], "amax", include_self=True)
    picked = torch.where(child >= 0, tok[child.clamp(min=0)], picked)
    state.update(tok=tok, picked=picked, free_pages=left,
                 top=torch.tensor([left.numel()], dtype=torch.int32, device=dev), ctx_len=empty(b),
                 free_top=empty(1), anchor=empty(b), mask=empty(rows, words, dtype=torch.int64),
                 pos=empty(rows), path=empty(b, GAMMA + 1), path_tok=empty(b, GAMMA),
                 accept_len=empty(b), out_tok=empty(b), committed=empty(b, GAMMA + 1),
                 n_committed=empty(b))
    if own:
        import speculative_decoding_verification_dspark_gb300 as dspark
        state["ws"] = empty(dspark.compact_workspace_size(b), dtype=torch.uint8)
    return state


def _prepare_sample(c, gen, dev):
    rows, v = c["b"] * c["per"], c["vocab"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    logits = torch.empty(rows, v + c["pad"], dtype=dt, device=dev)[:, :v]
    noise = torch.empty(rows, v, device=dev)
    step = max(1, (1 << 26) // v)
    for a in range(0, rows, step):
        z = min(rows, a + step)
        # a wide body, and in every row a few tokens that stand out by another amount
        x = 3 * torch.randn(z - a, v, generator=gen, device=dev)
        few = torch.randint(0, v, (z - a, 8), generator=gen, device=dev)
        lift = 14 * torch.rand(z - a, 1, generator=gen, device=dev)
        x.scatter_add_(1, few, lift * torch.rand(z - a, 8, generator=gen, device=dev))
        logits[a:z] = x.to(dt)
        u = torch.randint(0, 1 << 23, (z - a, v), generator=gen, device=dev)
        noise[a:z] = -torch.log((2 * u + 1).double() * 2.0 ** -24).float()  # no zero among them
    t, k, p, m = _params(c)
    f = dict(dtype=torch.float32, device=dev)
    state = {"case": c, "logits": logits, "noise": noise, "t": torch.tensor(t, **f),
             "k": torch.tensor(k, dtype=torch.int32, device=dev), "p": torch.tensor(p, **f),
             "m": torch.tensor(m, **f),
             "req": torch.arange(c["b"], dtype=torch.int32, device=dev).repeat_interleave(c["per"]),
             "tokens": torch.zeros(rows, dtype=torch.int32, device=dev), "probs": None}
    if c["probs"] != "none":
        state["probs"] = torch.zeros(rows, v, device=dev,
                                     dtype=torch.float32 if c["probs"] == "f32" else torch.bfloat16)
    return state


# ---------------------------------------------------------------- the operators
def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _own_attn, "sample": _own_sample, "tree": _own_tree}[op](state)
    return {"attn": _plain_attn, "sample": _plain_sample, "tree": _plain_tree}[op](state)


def _own_attn(s):
    import speculative_decoding_verification_dspark_gb300 as dspark
    dspark.verify_attn_tree(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"],
                            s["ctx"], s["cu"], s["mask"], s["scale"], 32, s["out"], s["lse"], s["ws"],
                            max_block_rows=s["width"])
    return s["out"], s["lse"]


def _own_sample(s):
    import speculative_decoding_verification_dspark_gb300 as dspark
    dspark.sample(s["logits"], s["t"], s["k"], s["p"], s["m"], s["noise"], s["tokens"], s["probs"],
                  row_req=s["req"])
    return (s["tokens"],) if s["probs"] is None else (s["tokens"], s["probs"])


def _own_tree(s):
    import speculative_decoding_verification_dspark_gb300 as dspark
    s["ctx_len"].copy_(s["ctx"])     # the lengths and the stack that the step finds
    s["free_top"].copy_(s["top"])
    dspark.tree_pack(s["parent"], s["cu"], s["ctx_len"], s["mask"], s["pos"])
    dspark.accept_tree(s["tok"], s["parent"], s["cu"], s["picked"], s["path"], s["path_tok"],
                       s["accept_len"], s["out_tok"])
    dspark.compact(s["k_new"], s["v_new"], s["cu"], s["accept_len"], s["out_tok"], s["path_tok"],
                   s["table"], s["ctx_len"], s["anchor"], s["free_pages"], s["free_top"],
                   s["k_cache"], s["v_cache"], s["committed"], s["n_committed"], s["ws"],
                   path=s["path"])
    return _tree_outputs(s)


def _tree_outputs(s):
    return tuple(s[k] for k in ("mask", "pos", "path", "accept_len", "out_tok", "ctx_len", "anchor",
                                "free_top", "table", "committed", "n_committed", "k_cache",
                                "v_cache"))


def _plain_attn(s):
    c, cu = s["case"], s["cu"].long()
    b, hq, hkv, n, dev = c["b"], c["hq"], c["hkv"], s["width"], s["cu"].device
    g, length = hq // hkv, s["length"]
    k, v = (x[s["table"].long()].flatten(1, 2)[:, :length].transpose(1, 2).float()
            for x in (s["k_cache"], s["v_cache"]))                      # [B, Hkv, L, 128]
    at = cu[:-1, None] + torch.arange(n, device=dev)                    # [B, n] packed rows
    live = at < cu[1:, None]
    at = at.clamp(max=s["rows"] - 1)
    q = s["q"][at].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    kn = s["k_new"][at].float().transpose(1, 2)
    vn = s["v_new"][at].float().transpose(1, 2)
    sc = torch.cat([q @ k.transpose(-1, -2), q @ kn.transpose(-1, -2)], -1).mul_(s["scale"])
    sc = sc.unflatten(2, (n, g))                                        # [B, Hkv, n, g, L + n]
    j = torch.arange(n, device=dev)
    bits = (s["mask"][at][..., j // 64] >> (j % 64)) & 1                # [B, n, n]
    old = (torch.arange(length, device=dev) < s["ctx"][:, None])[:, None].expand(b, n, length)
    seen = torch.cat([old, (bits > 0) & live[:, :, None] & live[:, None]], -1)
    sc = sc.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    e = sc.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(-1)
    w = e.div_(total.clamp(min=1e-30)).flatten(2, 3)
    o = (w[..., :length] @ v + w[..., length:] @ vn).unflatten(2, (n, g))
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[s["req"], s["i"]]
    lse = lse.permute(0, 2, 1, 3).flatten(2, 3)[s["req"], s["i"]]
    return o.to(torch.bfloat16), lse


def _plain_sample(s):
    """A row's tokens in order of their logits, the lowest index first among equals; each filter keeps
    a first part of that order.  In 64 bits, since the filters' borders and the race's winner hang on
    values that lie close together."""
    c, req = s["case"], s["req"].long()
    t, p, m = (s[x][req].double()[:, None] for x in ("t", "p", "m"))
    k, v = s["k"][req].long()[:, None], c["vocab"]
    greedy = t == 0
    value, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    z = (value - value[:, :1]) / torch.where(greedy, torch.ones_like(t), t)
    rank = torch.arange(v, device=z.device)
    keep = rank < torch.where(k > 0, k, torch.full_like(k, v))
    keep &= (z >= torch.log(m.clamp(min=0))) & (~greedy | (rank == 0))
    w = torch.where(keep, torch.exp(z), torch.zeros_like(z))
    before = torch.cumsum(w, 1) - w
    keep &= (before < p * w.sum(1, keepdim=True)) | (p >= 1)
    w = torch.where(keep, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order, w / w.sum(1, keepdim=True))
    score = w / s["noise"].double()
    best = score.max(1, keepdim=True).values
    tokens = (score == best).to(torch.uint8).argmax(1)     # the lowest index among the best
    tokens = torch.where(greedy[:, 0], order[:, 0], tokens).to(torch.int32)
    return (tokens,) if s["probs"] is None else (tokens, w.to(s["probs"].dtype))


def _plain_tree(s):
    c, cu = s["case"], s["cu"].long()
    b, dev, page, live = c["b"], cu.device, c["page"], s["req"].numel()
    sees = _ancestors(s["parent"], cu, s["req"], s["i"], 64 * s["words"])
    mask, pos = s["mask"].clone(), s["pos"].clone()
    mask[:live] = _words(sees)
    pos[:live] = (s["ctx"][s["req"]] + sees.sum(1) - 1).to(torch.int32)
    # a row is on the path where every step from the anchor down to it is: its token is the one that
    # its parent's row sampled, and no row before it says the same
    par, at = s["parent"][:live].long(), torch.arange(live, device=dev)
    up = (cu[s["req"]] + par).clamp(min=0)
    match = (par >= 0) & (s["tok"][:live] == s["picked"][up])
    first = torch.full((max(live, 1),), live, device=dev).scatter_reduce_(
        0, up[match], at[match], "amin", include_self=True)
    ok = (par < 0) & (s["i"] == 0) | match & (first[up] == at)
    off = (~ok).to(torch.float32)
    grid = torch.zeros(b, 64 * s["words"], device=dev)
    grid[s["req"], s["i"]] = off
    on = (sees.float() * grid[s["req"]]).sum(1) == 0
    depth = sees.sum(1) - 1
    on &= depth <= GAMMA
    path = torch.full((b, GAMMA + 1), -1, dtype=torch.int32, device=dev)
    path[s["req"][on], depth[on]] = s["i"][on].to(torch.int32)
    accept = ((path >= 0).sum(1) - 1).to(torch.int32)
    has = accept >= 0
    last = (cu[:-1] + path.gather(1, accept.clamp(min=0).long()[:, None])[:, 0]).clamp(min=0)
    out_tok = torch.where(has, s["picked"][last.clamp(max=s["rows"] - 1)], torch.full_like(accept, -1))
    # the commit: pages from the top of the stack, requests in order
    keep, ctx = accept + 1, s["ctx"]
    have, need = (ctx + page - 1) // page, (ctx + keep + page - 1) // page
    new = (need - have).long()
    start = torch.cumsum(new, 0) - new
    col = torch.arange(s["table"].shape[1], device=dev)
    nth = col - have[:, None]
    take = (nth >= 0) & (nth < new[:, None])
    src = (s["top"][0] - 1 - start[:, None] - nth).clamp(0, s["free_pages"].numel() - 1)
    table = torch.where(take, s["free_pages"][src], s["table"])
    r, d = s["req"][on], depth[on]
    to = ctx[r] + d
    where = table[r, (to // page).long()].long(), (to % page).long()
    s["k_cache"][where] = s["k_new"][:live][on]
    s["v_cache"][where] = s["v_new"][:live][on]
    committed = torch.full((b, GAMMA + 2), -1, dtype=torch.int32, device=dev)
    committed[r, torch.where(d > 0, d - 1, torch.full_like(d, GAMMA + 1))] = s["tok"][:live][on]
    committed[torch.arange(b, device=dev)[has], accept[has].long()] = out_tok[has]
    anchor = torch.where(has, out_tok, s["anchor"])
    return (mask, pos, path, accept, out_tok, ctx + keep, anchor, s["top"] - new.sum().to(torch.int32),
            table, committed[:, :GAMMA + 1], keep, s["k_cache"], s["v_cache"])


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    if case["op"] == "sample" and case["b"] * case["per"] > 600:
        return None     # row by row: too long
    s = prepare(case, seed)
    return {"attn": _exact_attn, "sample": _exact_sample, "tree": _exact_tree}[case["op"]](s)


def _parents_of(s, r):
    cu = s["cu"].tolist()
    return s["parent"].tolist()[cu[r]:cu[r + 1]]


def _chain(parents, j):
    """Row j and its ancestors, itself first."""
    out = []
    while j >= 0:
        out.append(j)
        j = parents[j]
    return out


def _exact_attn(s):
    """Request by request and node by node: the keys that the node's own way to the anchor gives."""
    c = s["case"]
    g, page, dev = c["hq"] // c["hkv"], c["page"], s["q"].device
    out = torch.zeros(s["rows"], c["hq"], D, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["rows"], c["hq"], dtype=torch.float64, device=dev)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    for r in range(c["b"]):
        a, z = cu[r], cu[r + 1]
        if a == z:
            continue
        parents = _parents_of(s, r)
        hidden = torch.ones(z - a, z - a, dtype=torch.bool)
        for j in range(z - a):
            hidden[j, _chain(parents, j)] = False
        hidden = hidden.to(dev).repeat_interleave(g, 0)
        ids = s["table"][r, :(ctx[r] + page - 1) // page].long()
        for h in range(c["hkv"]):
            k, v = (torch.cat([cache[ids, :, h].reshape(-1, D)[:ctx[r]], new[a:z, h]]).double()
                    for cache, new in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])))
            q = s["q"][a:z, h * g:(h + 1) * g].double().reshape(-1, D)
            sc = (q @ k.T) * s["scale"]
            sc[:, ctx[r]:][hidden] = -math.inf
            out[a:z, h * g:(h + 1) * g] = (torch.softmax(sc, -1) @ v).view(z - a, g, D)
            lse[a:z, h * g:(h + 1) * g] = torch.logsumexp(sc, -1).view(z - a, g)
    return out, lse


def _exact_sample(s):
    """Row by row over the distinct values of the logits: how many tokens of each value are kept, the
    last value's by their index."""
    c, dev = s["case"], s["logits"].device
    t, k, p, m = (s[x].tolist() for x in ("t", "k", "p", "m"))
    tokens, probs = [], []
    for row, r in enumerate(s["req"].tolist()):
        x = s["logits"][row].double()
        value, inverse, count = torch.unique(x, return_inverse=True, return_counts=True)
        if t[r] == 0:
            keep = torch.zeros_like(x, dtype=torch.bool)
            keep[(x == value[-1]).nonzero()[0, 0]] = True
            w = keep.double()
        else:
            each = torch.exp((value - value[-1]) / t[r]).flip(0)            # from the largest value
            num = torch.where((value.flip(0) - value[-1]) / t[r] >= (math.log(m[r]) if m[r] > 0 else -math.inf),
                              count.flip(0), torch.zeros_like(count))
            if k[r] > 0:
                num = torch.minimum(num, (k[r] - (num.cumsum(0) - num)).clamp(min=0))
            if p[r] < 1:
                mass = num * each
                before = mass.cumsum(0) - mass
                short = p[r] * mass.sum() - before
                num = torch.minimum(num, torch.ceil(short / each).clamp(min=0).nan_to_num().long())
            cls = value.numel() - 1 - inverse
            order = torch.argsort(cls, stable=True)
            place = torch.empty_like(order)
            place[order] = torch.arange(c["vocab"], device=dev)
            full = count.flip(0)
            nth = place - (full.cumsum(0) - full)[cls]                       # place among its equals
            w = torch.where(nth < num[cls], each[cls], torch.zeros_like(x))
            w = w / w.sum()
        race = torch.log(w) - torch.log(s["noise"][row].double())
        tokens.append((race == race.max()).nonzero()[0, 0])
        if s["probs"] is not None:
            probs.append(w)
    tokens = torch.stack(tokens).to(torch.int32)
    return (tokens,) if s["probs"] is None else (tokens, torch.stack(probs))


def _exact_tree(s):
    """The step's bookkeeping on the host, row by row."""
    c, cu = s["case"], s["cu"].tolist()
    page, tok, picked = c["page"], s["tok"].tolist(), s["picked"].tolist()
    mask, pos = s["mask"].cpu().clone(), s["pos"].cpu().clone()
    ctx, table = s["ctx"].tolist(), s["table"].cpu().clone()
    free, anchor = s["free_pages"].tolist(), s["anchor"].cpu().clone()
    path = torch.full((c["b"], GAMMA + 1), -1, dtype=torch.int32)
    committed = path.clone()
    accept, out_tok, from_rows, to_pages, to_slots = [], [], [], [], []
    for r in range(c["b"]):
        a, parents = cu[r], _parents_of(s, r)
        for j in range(len(parents)):
            line = _chain(parents, j)
            pos[a + j] = ctx[r] + len(line) - 1
            word = [0] * s["words"]
            for q in line:
                word[q // 64] |= 1 << (q % 64)
            mask[a + j] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in word])
        at, way = 0, []
        while parents and at is not None:
            way.append(at)
            say = picked[a + at]
            at = next((j for j in range(len(parents)) if parents[j] == at and tok[a + j] == say), None)
            if len(way) == GAMMA + 1:
                at = None
        accept.append(len(way) - 1)
        out_tok.append(picked[a + way[-1]] if way else -1)
        for d, j in enumerate(way):
            path[r, d] = j
            if (ctx[r] + d) % page == 0:
                table[r, (ctx[r] + d) // page] = free.pop()
            from_rows.append(a + j)
            to_pages.append(int(table[r, (ctx[r] + d) // page]))
            to_slots.append((ctx[r] + d) % page)
            committed[r, d] = tok[a + way[d + 1]] if d + 1 < len(way) else out_tok[-1]
        ctx[r] += len(way)
        if way:
            anchor[r] = out_tok[-1]
    k, v = s["k_cache"].double(), s["v_cache"].double()
    k[to_pages, to_slots] = s["k_new"][from_rows].double()
    v[to_pages, to_slots] = s["v_new"][from_rows].double()
    i32 = dict(dtype=torch.int32)
    whole = (mask, pos, path, torch.tensor(accept, **i32), torch.tensor(out_tok, **i32),
             torch.tensor(ctx, **i32), anchor, torch.tensor([len(free)], **i32), table, committed,
             torch.tensor(accept, **i32) + 1)
    return tuple(x.to(k.device) for x in whole) + (k, v)
