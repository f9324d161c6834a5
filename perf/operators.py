"""Measured cases of the query/key norm with position rotation and of the 4-bit KV cache:
their inputs, their plain forms in elementary torch operations, the framework's calls,
and their definitions in 64 bits.

A 4-bit cache page holds, for each KV head and 16 tokens, one block of 2176 bytes:
K codes [4 groups of 32 dims][16 tokens][16 B], V codes [128 channels][8 B], K scales
[16 tokens][4 groups] and V scales [4 groups][16 tokens] (e4m3).  In every 32-bit word of
codes, nibble p holds element 2p and nibble p + 4 element 2p + 1 of eight consecutive
ones (dims of a token for K, tokens of a channel for V).  value = (code - 8) * scale * g
with one fp32 factor g per tensor.
"""
import math

import torch

own = False

D = 128            # head dim
GROUP = 32         # elements that share a scale
BLOCK = 16         # tokens of a block
BLOCK_BYTES = 2176
K_SCALE, V_SCALE = 1.0 / 32, 0.0317  # a power of two and a calibrated factor
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _rope(name, rows, tier, hq, hkv, rotary, interleaved, dtype, fused, max_pos):
    return {"name": name, "op": "norm_rope", "rows": rows, "tier": tier, "hq": hq, "hkv": hkv,
            "rotary": rotary, "interleaved": interleaved, "dtype": dtype, "fused": fused,
            "max_pos": max_pos}


def _kv4(name, b, n_lo, n_hi, p_lo, p_hi, hkv, page, dtype):
    return {"name": name, "op": "kv4", "b": b, "n_lo": n_lo, "n_hi": n_hi, "p_lo": p_lo,
            "p_hi": p_hi, "hkv": hkv, "page": page, "dtype": dtype}


def _attn(name, b, n_lo, n_hi, c_lo, c_hi, hq, hkv, page):
    return {"name": name, "op": "attn", "b": b, "n_lo": n_lo, "n_hi": n_hi, "c_lo": c_lo,
            "c_hi": c_hi, "hq": hq, "hkv": hkv, "page": page}


def listed():
    return [
        # one token of one request on its way into the attention: latency alone
        _rope("rope_one_token", 1, 1, 32, 8, 128, False, "bf16", True, 4096),
        # the rows of a compact verification step, padded to the captured tier
        _rope("rope_verify_tier", 174, 256, 32, 8, 128, False, "bf16", True, 4104),
        # a prompt chunk with positions far out
        _rope("rope_prompt", 16384, 16384, 40, 8, 128, False, "bf16", True, 131072),
        # half of each head rotated in adjacent pairs, fp32 projections, an odd row count
        _rope("rope_partial_f32", 4099, 4099, 8, 2, 64, True, "f32", False, 1000000),
        # the accepted rows of a step appended in the middle of blocks
        _kv4("kv4_commit", 32, 1, 9, 1024, 4096, 8, 16, "bf16"),
        # prompts of ragged lengths, fp32 rows, few heads
        _kv4("kv4_ragged_f32", 8, 1, 4099, 0, 700, 2, 64, "f32"),
        # long prompts
        _kv4("kv4_prompt", 4, 16384, 16384, 0, 0, 8, 16, "bf16"),
        # one token of one request
        _attn("attn_one_token", 1, 1, 1, 997, 997, 32, 8, 16),
        # a compact verification step: short ragged windows
        _attn("attn_verify", 32, 1, 9, 1024, 4096, 32, 8, 16),
        # many requests that decode single tokens
        _attn("attn_decode_wide", 256, 1, 1, 512, 4096, 40, 8, 16),
        # whole blocks verified, as in static and cap-accept mode
        _attn("attn_block", 64, 17, 17, 2048, 2048, 32, 8, 64),
        # few requests with long contexts
        _attn("attn_long", 3, 3, 7, 131071, 131071, 40, 8, 64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("norm_rope", "kv4", "attn", "attn"))
    hq, hkv = rng.choice(((8, 2), (20, 4), (32, 8), (40, 8), (32, 4), (16, 16), (7, 1)))
    if op == "norm_rope":
        rows = _log(rng, 1, 10000)
        c = _rope("", rows, rows + rng.choice((0, 0, 1, 13, 64)), hq, hkv,
                  rng.choice((128, 128, 64, 96, 32)), rng.random() < 0.4,
                  rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.6,
                  _log(rng, 1000, 1000000))
    elif op == "kv4":
        b = _log(rng, 1, 200)
        hi = _log(rng, 1, max(1, 20000 // b))
        p = _log(rng, 1, 2000)
        c = _kv4("", b, rng.randint(1, hi), hi, rng.randint(0, p), p, hkv,
                 rng.choice((16, 16, 32, 64, 128)), rng.choice(("bf16", "bf16", "f32")))
    else:
        b = _log(rng, 1, 190)
        hi = _log(rng, 1, min(100000, 240000 // b))
        n = rng.choice((1, 1, rng.randint(2, 9), rng.randint(2, 17)))
        n = min(n, max(1, 1500 // b))
        c = _attn("", b, rng.randint(1, n), n, rng.randint(hi // 3, hi), hi, hq, hkv,
                  rng.choice((16, 16, 32, 64, 128)))
    del c["name"]
    return c


def _spread(lo, hi, b):
    """b lengths over [lo, hi], the same for every seed: a case's work is its own."""
    return [lo + (i * 7919 + 13) % (hi - lo + 1) for i in range(b)]


def _lengths(c):
    """(row counts, positions of the first rows) of a case's requests."""
    if c["op"] == "kv4":
        return _spread(c["n_lo"], c["n_hi"], c["b"]), _spread(c["p_lo"], c["p_hi"], c["b"])
    return _spread(c["n_lo"], c["n_hi"], c["b"]), _spread(c["c_lo"], c["c_hi"], c["b"])


def work(case):
    c = case
    if c["op"] == "norm_rope":
        heads, s = c["hq"] + 2 * c["hkv"], 2 if c["dtype"] == "bf16" else 4
        n = c["rows"] * heads * D
        return {"bytes": n * (s + 2) + 4 * c["tier"], "flops": 10.0 * n}
    n, p = _lengths(c)
    if c["op"] == "kv4":
        s = 2 if c["dtype"] == "bf16" else 4
        rows = sum(n) * c["hkv"]
        # rows in, codes and scales out, those in again and bf16 rows out
        return {"bytes": rows * 2.0 * (D * s + 68 + 68 + D * 2), "flops": rows * 2.0 * D * 6}
    rows, keys = sum(n), 0
    for a, b in zip(n, p):
        keys += a * b + a * (a + 1) // 2
    by = sum(p) * c["hkv"] * 136.0 + rows * ((c["hq"] + 2 * c["hkv"]) * D * 2 + c["hq"] * (D * 2 + 4))
    return {"bytes": by, "flops": 4.0 * keys * c["hq"] * D}


# ---------------------------------------------------------------- inputs
def _e4m3_at_least(t):
    """The smallest e4m3 number >= t (t >= 0; 448 above it), as (code, value)."""
    t = t.clamp(max=448.0)
    s = t.to(torch.float8_e4m3fn)
    code = s.view(torch.uint8)
    code = torch.where(s.float() < t, code + 1, code)
    return code, code.view(torch.float8_e4m3fn).float()


def _quantise(x, g):
    """x fp32 [..., 128] -> (codes 1..15 [..., 128], scale codes [..., 4], values [..., 128])."""
    xg = x.unflatten(-1, (D // GROUP, GROUP))
    code, s = _e4m3_at_least(xg.abs().amax(-1) / (x.new_tensor(7.0) * g))
    sg = (s * g).unsqueeze(-1)
    q = torch.where(sg > 0, xg / sg, torch.zeros_like(xg)).round().clamp(-7, 7)
    return (q + 8).flatten(-2), code, (q * s.unsqueeze(-1) * g).flatten(-2)


def _nibbles(codes):
    """codes [..., 8m] -> bytes [..., 4m]."""
    c = codes.to(torch.uint8).unflatten(-1, (-1, 4, 2)).transpose(-1, -2)  # [m, half, p]
    c = c.flatten(-2).unflatten(-1, (4, 2))                                # nibble = 2 byte + high
    return (c[..., 0] | (c[..., 1] << 4)).flatten(-2)


def _blocks(k, v):
    """k, v fp32 [n, 16, 128] (tokens of n blocks) -> bytes [n, 2176]."""
    n = k.shape[0]
    kc, ks, _ = _quantise(k, K_SCALE)
    vc, vs, _ = _quantise(v, V_SCALE)
    kb = _nibbles(kc).view(n, BLOCK, 4, 16).transpose(1, 2).reshape(n, 1024)
    vb = _nibbles(vc.transpose(1, 2)).reshape(n, 1024)
    return torch.cat([kb, vb, ks.reshape(n, 64), vs.transpose(1, 2).reshape(n, 64)], 1)


def _fill_cache(n_pages, hkv, page, gen, dev):
    """A pool of pages with quantised keys (some channels larger, as after a per-head norm
    with learned weights) and values."""
    per = page // BLOCK
    cache = torch.empty(n_pages, hkv, per, BLOCK_BYTES, dtype=torch.uint8, device=dev)
    gain = torch.exp(0.5 * torch.randn(hkv, 1, D, generator=gen, device=dev))
    step = max(1, 8192 // (hkv * per))
    for a in range(0, n_pages, step):
        m = min(step, n_pages - a)
        k = torch.randn(m, hkv, per * BLOCK, D, generator=gen, device=dev)
        k = (k * gain).reshape(-1, BLOCK, D)
        v = 0.5 * torch.randn(m * hkv * per, BLOCK, D, generator=gen, device=dev)
        cache[a:a + m] = _blocks(k, v).view(m, hkv, per, BLOCK_BYTES)
    return cache


def _pages(tokens, page, gen, dev):
    """A table of distinct pages in random order for requests of these token counts."""
    need = [(t + page - 1) // page for t in tokens]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    width = max(max(need), 1)
    col = torch.arange(width, device=dev)
    cnt = torch.tensor(need, device=dev)
    first = torch.cumsum(cnt, 0) - cnt
    at = (first[:, None] + col).clamp(max=n_pages - 1)
    return torch.where(col < cnt[:, None], perm[at], torch.zeros_like(perm[at])), n_pages


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 1000003 + 17)
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    hkv = c["hkv"]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if c["op"] == "norm_rope":
        hq, rows, tier = c["hq"], c["rows"], c["tier"]
        parts = [(2 * rand(tier, h, D)).to(dt) for h in (hq, hkv, hkv)]
        if c["fused"]:  # one projection's output, its parts side by side in each row
            qkv = torch.cat([p.flatten(1) for p in parts], 1)
            parts = [p.unflatten(1, (-1, D)) for p in qkv.split([hq * D, hkv * D, hkv * D], 1)]
        pos = torch.randint(0, c["max_pos"], (tier,), generator=gen, device=dev, dtype=torch.int32)
        pos[rows:] = -1
        inv = 10.0 ** (-6.0 * torch.arange(0, c["rotary"], 2, device=dev, dtype=torch.float64) / c["rotary"])
        return {"case": c, "q_in": parts[0], "k_in": parts[1], "v_in": parts[2], "pos": pos,
                "wq": 1 + 0.2 * rand(D), "wk": 1 + 0.2 * rand(D), "inv_freq": inv.float(),
                "q": torch.zeros(tier, hq, D, dtype=torch.bfloat16, device=dev),
                "k": torch.zeros(tier, hkv, D, dtype=torch.bfloat16, device=dev),
                "v": torch.zeros(tier, hkv, D, dtype=torch.bfloat16, device=dev)}

    n, p = _lengths(c)
    cu = torch.tensor([0] + n, device=dev).cumsum(0).to(torch.int32)
    first = torch.tensor(p, device=dev, dtype=torch.int32)
    rows = sum(n)
    req = torch.repeat_interleave(torch.arange(c["b"], device=dev), torch.tensor(n, device=dev))
    state = {"case": c, "cu": cu, "first": first, "req": req, "rows": rows,
             "i": torch.arange(rows, device=dev) - cu[req]}
    if c["op"] == "kv4":
        table, n_pages = _pages([a + b for a, b in zip(n, p)], c["page"], gen, dev)
        state.update(table=table, k=rand(rows, hkv, D).to(dt), v=(0.5 * rand(rows, hkv, D)).to(dt),
                     cache=torch.zeros(n_pages, hkv, c["page"] // BLOCK, BLOCK_BYTES,
                                       dtype=torch.uint8, device=dev),
                     k_out=torch.zeros(rows, hkv, D, dtype=torch.bfloat16, device=dev),
                     v_out=torch.zeros(rows, hkv, D, dtype=torch.bfloat16, device=dev))
        return state
    hq = c["hq"]
    table, n_pages = _pages(p, c["page"], gen, dev)
    bf = torch.bfloat16
    state.update(table=table, cache=_fill_cache(n_pages, hkv, c["page"], gen, dev),
                 q=(1.5 * rand(rows, hq, D)).to(bf), k_new=rand(rows, hkv, D).to(bf),
                 v_new=(0.5 * rand(rows, hkv, D)).to(bf),
                 n_max=max(n), blocks=(max(p) + BLOCK - 1) // BLOCK, scale=1.0 / math.sqrt(D),
                 out=torch.zeros(rows, hq, D, dtype=bf, device=dev),
                 lse=torch.zeros(rows, hq, dtype=torch.float32, device=dev))
    if own:  # the workspace that a serving program keeps for its steps
        import speculative_decoding_verification_dspark_gb300 as dspark
        state["hint"] = dspark.block_rows_hint_for_kv4(max(n) - 1, hq, hkv)
        state["ws"] = torch.empty(dspark.verify_attn_kv4_workspace_size(
            c["b"], rows, hq, hkv, 32, state["hint"]), dtype=torch.uint8, device=dev)
    return state


# ---------------------------------------------------------------- the operators
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_rope": _own_rope, "kv4": _own_kv4, "attn": _own_attn}[op](state)
    return {"norm_rope": _plain_rope, "kv4": _plain_kv4, "attn": _plain_attn}[op](state)


def _own_rope(s):
    import speculative_decoding_verification_dspark_gb300 as dspark
    dspark.qk_norm_rope(s["q_in"], s["k_in"], s["v_in"], s["wq"], s["wk"], s["inv_freq"], s["pos"],
                        s["q"], s["k"], s["v"], eps=EPS, interleaved=s["case"]["interleaved"])
    return s["q"], s["k"], s["v"]


def _own_kv4(s):
    import speculative_decoding_verification_dspark_gb300 as dspark
    dspark.kv4_store(s["k"], s["v"], s["cu"], s["first"], s["table"], s["cache"], K_SCALE, V_SCALE)
    dspark.kv4_load(s["cache"], s["cu"], s["first"], s["table"], s["k_out"], s["v_out"], K_SCALE,
                    V_SCALE)
    return s["k_out"], s["v_out"]


def _own_attn(s):
    import speculative_decoding_verification_dspark_gb300 as dspark
    dspark.verify_attn_kv4(s["q"], s["k_new"], s["v_new"], s["cache"], s["table"], s["first"],
                           s["cu"], s["scale"], 32, s["out"], s["lse"], s["ws"], K_SCALE, V_SCALE,
                           max_block_rows=s["hint"])
    return s["out"], s["lse"]


def _plain_norm_rope(x, w, c, cos, sin):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    half = c["rotary"] // 2
    if c["interleaved"]:
        a, b = y[..., 0:c["rotary"]:2], y[..., 1:c["rotary"]:2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:c["rotary"]]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, y[..., c["rotary"]:]], -1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    # positions reach 10^6: the angles in 64 bits
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    live = (s["pos"] >= 0)[:, None, None]
    q = torch.where(live, _plain_norm_rope(s["q_in"], s["wq"], c, cos, sin), s["q"])
    k = torch.where(live, _plain_norm_rope(s["k_in"], s["wk"], c, cos, sin), s["k"])
    return q, k, torch.where(live, s["v_in"].to(torch.bfloat16), s["v"])


def _plain_kv4(s):
    return (_quantise(s["k"].float(), K_SCALE)[2].to(torch.bfloat16),
            _quantise(s["v"].float(), V_SCALE)[2].to(torch.bfloat16))


def _codes(b):
    """bytes [..., 4m] -> codes - 8 [..., 8m] fp32."""
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2)                  # nibble order
    return c.unflatten(-1, (-1, 2, 4)).transpose(-1, -2).flatten(-3).float() - 8.0


def _plain_cache(s):
    """K and V of every request's committed positions, fp32 [B, Hkv, L, 128]."""
    c, nb = s["case"], s["blocks"]
    per = c["page"] // BLOCK
    x = s["cache"][s["table"].long()]                                   # [B, pages, Hkv, per, 2176]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :max(nb, 1)]       # [B, Hkv, blocks, 2176]
    ks = x[..., 2048:2112].view(torch.float8_e4m3fn).float().unflatten(-1, (BLOCK, 4))
    k = _codes(x[..., :1024].unflatten(-1, (4, BLOCK, 16))).transpose(-2, -3)   # [.., tok, grp, 32]
    k = (k * ks[..., None] * K_SCALE).flatten(-2).flatten(2, 3)
    vs = x[..., 2112:].view(torch.float8_e4m3fn).float().unflatten(-1, (4, 1, BLOCK))
    v = _codes(x[..., 1024:2048].unflatten(-1, (4, GROUP, 8)))          # [.., grp, ch, tok]
    v = (v * vs * V_SCALE).flatten(-3, -2).transpose(-1, -2).flatten(2, 3)
    return k, v


def _plain_attn(s):
    c, cu = s["case"], s["cu"].long()
    b, hq, hkv, n = c["b"], c["hq"], c["hkv"], s["n_max"]
    g = hq // hkv
    k, v = _plain_cache(s)
    length = k.shape[2]
    at = cu[:-1, None] + torch.arange(n, device=cu.device)              # [B, n] packed rows
    live = at < cu[1:, None]
    at = at.clamp(max=s["rows"] - 1)
    q = s["q"][at].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    kn = s["k_new"][at].float().transpose(1, 2)
    vn = s["v_new"][at].float().transpose(1, 2)
    sc = torch.cat([q @ k.transpose(-1, -2), q @ kn.transpose(-1, -2)], -1) * s["scale"]
    sc = sc.unflatten(2, (n, g))                                        # [B, Hkv, n, g, L + n]
    i = torch.arange(n, device=cu.device)
    seen = torch.cat([(torch.arange(length, device=cu.device) < s["first"][:, None])[:, None].expand(b, n, length),
                      live[:, None] & (i[None, None] <= i[None, :, None])], -1)
    sc = sc.masked_fill(~seen[:, None, :, None], -math.inf)
    top = sc.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(sc - top)
    total = e.sum(-1, keepdim=True)
    w = (e / total).flatten(2, 3)
    o = (w[..., :length] @ v + w[..., length:] @ vn).unflatten(2, (n, g))
    lse = (top + torch.log(total)).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)[s["req"], s["i"]]
    lse = lse.permute(0, 2, 1, 3).flatten(2, 3)[s["req"], s["i"]]
    return o.to(torch.bfloat16), lse


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _exact_rope, "kv4": _exact_kv4, "attn": _exact_attn}[case["op"]](s)


def _exact_rope(s):
    """The rotation as a product of complex numbers."""
    c, r = s["case"], s["case"]["rotary"]
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=s["pos"].device),
                       torch.outer(s["pos"].double(), s["inv_freq"].double()))[:, None]

    def one(x, w, before):
        x = x.double()
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w.double()
        h = y[..., :r].unflatten(-1, (r // 2, 2) if c["interleaved"] else (2, r // 2))
        ax = -1 if c["interleaved"] else -2
        z = torch.complex(h.select(ax, 0), h.select(ax, 1)) * turn
        y = torch.cat([torch.stack([z.real, z.imag], ax).flatten(-2), y[..., r:]], -1)
        y[s["pos"] < 0] = before[s["pos"] < 0].double()
        return y

    v = s["v_in"].double().clone()
    v[s["pos"] < 0] = s["v"][s["pos"] < 0].double()
    return one(s["q_in"], s["wq"], s["q"]), one(s["k_in"], s["wk"], s["k"]), v


def _exact_kv4(s):
    every = torch.arange(127, dtype=torch.uint8, device=s["k"].device).view(torch.float8_e4m3fn).double()

    def one(x, g):
        x = x.double().unflatten(-1, (-1, GROUP))
        top = x.abs().max(-1, keepdim=True).values
        scale = every[torch.searchsorted(every, (top / (7 * g)).contiguous()).clamp(max=126)] * g
        q = torch.nan_to_num(torch.round(x / scale)).clamp(-7, 7)
        return (q * scale).flatten(-2)

    g = lambda f: float(torch.tensor(f, dtype=torch.float32))  # noqa: E731
    return one(s["k"], g(K_SCALE)), one(s["v"], g(V_SCALE))


def _exact_attn(s):
    c = s["case"]
    g, page, dev = c["hq"] // c["hkv"], c["page"], s["q"].device
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=dev)  # element held by each nibble
    place = torch.argsort(order)
    g_k, g_v = (float(torch.tensor(f, dtype=torch.float32)) for f in (K_SCALE, V_SCALE))
    out = torch.zeros(s["rows"], c["hq"], D, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["rows"], c["hq"], dtype=torch.float64, device=dev)
    cu, first = s["cu"].tolist(), s["first"].tolist()

    def eights(b):
        word = b.reshape(*b.shape[:-1], -1, 4).to(torch.int64)
        word = word[..., 0] | word[..., 1] << 8 | word[..., 2] << 16 | word[..., 3] << 24
        nib = (word[..., None] >> (4 * torch.arange(8, device=dev))) & 15
        return (nib[..., place] - 8).flatten(-2)

    for r in range(c["b"]):
        a, z, ctx = cu[r], cu[r + 1], first[r]
        x = s["cache"][s["table"][r, :(ctx + page - 1) // page].long()]       # [pages, Hkv, per, 2176]
        for h in range(c["hkv"]):
            y = x[:, h].reshape(-1, BLOCK_BYTES)
            nb = y.shape[0]
            ks = y[:, 2048:2112].reshape(nb, BLOCK, 4, 1).view(torch.float8_e4m3fn).double()
            vs = y[:, 2112:].reshape(nb, 4, BLOCK, 1).view(torch.float8_e4m3fn).double()
            k = eights(y[:, :1024].reshape(nb, 4, BLOCK, 16)).permute(0, 2, 1, 3) * ks * g_k
            v = eights(y[:, 1024:2048].reshape(nb, 4, GROUP, 8)).permute(0, 1, 3, 2) * vs * g_v
            k = torch.cat([k.reshape(-1, D)[:ctx], s["k_new"][a:z, h].double()])
            v = torch.cat([v.permute(0, 2, 1, 3).reshape(-1, D)[:ctx], s["v_new"][a:z, h].double()])
            q = s["q"][a:z, h * g:(h + 1) * g].double().reshape(-1, D)
            sc = (q @ k.T) * s["scale"]
            row = torch.arange(z - a, device=dev).repeat_interleave(g)
            col = torch.arange(k.shape[0], device=dev) - ctx
            sc[col[None] > row[:, None]] = -math.inf
            out[a:z, h * g:(h + 1) * g] = (torch.softmax(sc, -1) @ v).view(z - a, g, D)
            lse[a:z, h * g:(h + 1) * g] = torch.logsumexp(sc, -1).view(z - a, g)
    return out, lse
