"""Verify attention over the 4-bit cache (dspark_verify_attn_kv4) against the softmax of
its definition in fp64 on the values the cache stands for, and its refusals.

Tolerance, from the arithmetic (S = max over a row's keys of scale * sum |q k|, A = the
weighted sum of |v|, n the row's keys):
  * a score is a sum of 128 products, exact in the fp16 operands, accumulated in fp32 (each
    step off by at most 2^-23): 128 * 2^-23 S; its scaling and the exponential's argument
    add 8 * 2^-23 S, the exponential 2^-21; a block row's key is rounded to fp16 (2^-11):
    2^-11 of the S over block rows.  Together es; a weight is off by 2 es relative (its own
    and the normaliser's).
  * probabilities and block rows' values are rounded to fp16: 2^-11 each, and a
    probability under fp16's range by 2^-25 of the largest.
  * sums over n keys in fp32: n 2^-23, and a merge of split pieces 64 * 2^-23.
  * the output's own rounding to bf16: 2^-8 of the value.
The lse is off by es and the sums."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import speculative_decoding_verification_dspark_gb300 as p
    return p


# ------------------------------------------------------------------ refusals (CPU)
def test_host_refusals(pkg):
    lib, f, off = pkg.load(), ctypes.c_void_p(4096), ctypes.c_void_p(4104)

    def call(q=f, c=f, gk=1.0, gv=1.0, tab=f, ctx=f, cu=f, B=2, rows=8, hq=8, hkv=2, page=16,
             scale=0.1, splits=8, hint=4, out=f, lse=f, ws=f, n=1 << 30,
             pages=9):
        return lib.dspark_verify_attn_kv4(q, f, f, c, gk, gv, pages, tab, 4, ctx, cu, B, rows, hq, hkv, page,
                                  ctypes.c_float(scale), splits, hint, out, lse, ws, n, None)

    for bad in (dict(q=None), dict(c=None), dict(tab=None), dict(ctx=None), dict(cu=None),
                dict(out=None), dict(lse=None), dict(ws=None), dict(q=off), dict(c=off),
                dict(out=off), dict(ws=off), dict(gk=0.0), dict(gv=float("nan")), dict(B=0),
                dict(B=1025), dict(rows=0), dict(scale=0.0), dict(scale=float("nan")),
                dict(splits=0), dict(splits=33)):
        assert call(**bad) == -1, bad
    for bad in (dict(hq=9), dict(hq=66), dict(hkv=0), dict(page=8), dict(page=40),
                dict(page=64, pages=1 << 28), dict(page=1 << 30, pages=1 << 5)):
        assert call(**bad) == -2, bad
    size = lib.dspark_verify_attn_kv4_workspace_size
    assert size(2, 8, 9, 2, 8, 4) == 0 and size(0, 8, 8, 2, 8, 4) == 0 and size(2, 8, 66, 2, 8, 1) == 0
    assert size(32, 512, 32, 8, 8, 0) == size(32, 512, 32, 8, 8, 2) > 0
    assert size(32, 512, 32, 8, 8, 16) == size(32, 512, 32, 8, 8, 99) > 0


def test_hint_and_binding_refusals(pkg):
    assert pkg.block_rows_hint_for_kv4(6, 32, 8) == 7
    assert pkg.block_rows_hint_for_kv4(16, 32, 8) == 9      # 17 rows in two tiles
    assert pkg.block_rows_hint_for_kv4(32, 32, 8) == 11     # 33 rows in three
    assert pkg.block_rows_hint_for_kv4(6, 64, 2) == 2       # 7 rows in four
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    c = pkg.kv4_cache(4, 2, 16, device="cpu")
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError):      # host tensors
        pkg.verify_attn_kv4(b(3, 8, 128), b(3, 2, 128), b(3, 2, 128), c, i(2, 4), i(2), i(3), 0.1, 8,
                            b(3, 8, 128), torch.zeros(3, 8), ws)
    with pytest.raises(ValueError):
        pkg.VerifyStep(2, 4, 128, 1, 576, 512, 1024, 16, device="cpu", kv4=True)


# ------------------------------------------------------------------ parity (GPU)
def _case(ctx, lens, hq, hkv, page, seed=0, qstd=1.0, tail=0, gk=0.0625, gv=0.0173, std=(1.0, 0.5)):
    """Random codes and scales; positions from ctx on hold NaN scales."""
    g = torch.Generator().manual_seed(seed)
    B, M = len(ctx), sum(lens)
    need = [-(-c // page) for c in ctx]
    n_pages = sum(need) + 2
    cache = torch.randint(0, 256, (n_pages, hkv, page // 16, O.KV4_BLOCK_BYTES), generator=g,
                          dtype=torch.uint8)
    # scales about std / (4 g): codes are uniform over -8..7
    for a, z, s, f in ((2048, 2112, std[0], gk), (2112, 2176, std[1], gv)):
        sc = s / 4.6 / f * torch.exp(0.4 * torch.randn(*cache.shape[:3], z - a, generator=g))
        cache[..., a:z] = sc.clamp(2 ** -9, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((B, max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
        for pos in range(ctx[r], n * page):
            blk = cache[int(table[r, pos // page]), :, pos % page // 16]
            blk[:, 2048 + pos % 16 * 4:2048 + pos % 16 * 4 + 4] = 0x7f
            blk[:, 2112 + pos % 16::16] = 0x7f
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    q = (qstd * torch.randn(M + tail, hq, 128, generator=g)).bfloat16()
    kn = (std[0] * torch.randn(M + tail, hkv, 128, generator=g)).bfloat16()
    vn = (std[1] * torch.randn(M + tail, hkv, 128, generator=g)).bfloat16()
    if tail:
        q[M:], kn[M:], vn[M:] = float("nan"), float("nan"), float("nan")
    return dict(q=q, k_new=kn, v_new=vn, cache=cache, table=table, cu=cu, gk=gk, gv=gv,
                ctx=torch.tensor(ctx, dtype=torch.int32), hq=hq, hkv=hkv, page=page, M=M,
                scale=1.0 / np.sqrt(128))


def _reference(c):
    """o, lse and their tolerances in fp64."""
    K, V = O.kv4_values(c["cache"].numpy(), c["gk"], c["gv"])
    q, kn, vn = (c[k].double().numpy() for k in ("q", "k_new", "v_new"))
    G, M = c["hq"] // c["hkv"], c["M"]
    o = np.zeros((M, c["hq"], 128))
    lse = np.zeros((M, c["hq"]))
    to, tl = np.zeros_like(o), np.zeros_like(lse)
    cu, table = c["cu"].tolist(), c["table"].numpy()
    e23 = 2.0 ** -23
    for r, ctx in enumerate(c["ctx"].tolist()):
        a, z = cu[r], cu[r + 1]
        pages = table[r, :-(-ctx // c["page"])]
        for h in range(c["hkv"]):
            k = np.concatenate([K[pages, :, h].reshape(-1, 128)[:ctx], kn[a:z, h]])
            v = np.concatenate([V[pages, :, h].reshape(-1, 128)[:ctx], vn[a:z, h]])
            for i in range(z - a):
                n = ctx + i + 1
                x = q[a + i, h * G:(h + 1) * G]
                s = c["scale"] * x @ k[:n].T
                S = c["scale"] * np.abs(x) @ np.abs(k[:n]).T
                m = s.max(-1, keepdims=True)
                w = np.exp(s - m)
                l = w.sum(-1, keepdims=True)
                w /= l
                sl = slice(h * G, (h + 1) * G)
                o[a + i, sl] = w @ v[:n]
                lse[a + i, sl] = (m + np.log(l))[:, 0]
                es = 136 * e23 * S.max(-1) + 2.0 ** -11 * S[:, ctx:].max(-1) + 2.0 ** -21
                acc = (n + 64) * e23
                A = w @ np.abs(v[:n])
                to[a + i, sl] = (2.0 ** -8 * np.abs(o[a + i, sl])
                                 + A * (2.0 ** -10 + 2 * es[:, None] + acc)
                                 + n * 2.0 ** -25 * np.abs(v[:n]).max(0))
                tl[a + i, sl] = es + acc + e23 * np.abs(lse[a + i, sl])
    return o, lse, to, tl


def _run(pkg, c, hint=None, splits=8, stream=None, ws=None, tail_fill=5.0):
    d = {k: c[k].cuda() for k in ("q", "k_new", "v_new", "cache", "table", "cu", "ctx")}
    rows, B = c["q"].shape[0], len(c["ctx"])
    if hint is None:
        hint = pkg.block_rows_hint_for_kv4(max(np.diff(c["cu"].numpy())) - 1, c["hq"], c["hkv"])
    out = torch.full((rows, c["hq"], 128), tail_fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows, c["hq"]), tail_fill, device="cuda")
    if ws is None:
        ws = torch.empty(pkg.verify_attn_kv4_workspace_size(B, rows, c["hq"], c["hkv"], splits, hint),
                         dtype=torch.uint8, device="cuda")
    call = lambda: pkg.verify_attn_kv4(  # noqa: E731
        d["q"], d["k_new"], d["v_new"], d["cache"], d["table"], d["ctx"], d["cu"], c["scale"],
        splits, out, lse, ws, c["gk"], c["gv"], stream, max_block_rows=hint)
    return call, out, lse


def _check(c, out, lse, tail_fill=5.0):
    o, l, to, tl = _reference(c)
    M = c["M"]
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got[:M]).all() and np.isfinite(gl[:M]).all()
    bad = np.abs(got[:M] - o) - to
    assert bad.max() <= 0, (np.unravel_index(bad.argmax(), bad.shape), bad.max())
    bad = np.abs(gl[:M] - l) - tl
    assert bad.max() <= 0, (np.unravel_index(bad.argmax(), bad.shape), bad.max())
    assert (got[M:] == tail_fill).all() and (gl[M:] == tail_fill).all()


SHAPES = [  # ctx, lens, hq, hkv, page
    ([0], [1], 1, 1, 16),
    ([1], [1], 4, 1, 16),
    ([0, 0], [5, 1], 8, 2, 16),
    ([15, 16, 17, 127, 128, 129], [1, 2, 3, 1, 5, 9], 8, 2, 16),
    ([255, 256, 257, 31, 33], [9, 1, 4, 0, 7], 32, 8, 16),
    ([300, 5, 1000, 640], [17, 17, 17, 17], 8, 2, 64),
    ([200, 700], [6, 3], 40, 8, 32),
    ([513, 90], [4, 2], 7, 1, 256),
    ([140, 300], [3, 1], 32, 1, 16),
    ([260, 0, 60], [33, 20, 1], 6, 2, 16),
    ([77, 130], [150, 140], 4, 4, 16),
    ([2500], [3], 16, 2, 128),
    ([1700, 3, 900], [16, 12, 15], 8, 2, 16),             # 64 query rows to a tile
    ([130, 640], [64, 33], 2, 2, 32),
    ([40] * 50, [1] * 50, 4, 2, 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,lens,hq,hkv,page", SHAPES)
@pytest.mark.parametrize("qstd", [1.0, 6.0])
def test_parity(pkg, ctx, lens, hq, hkv, page, qstd):
    c = _case(ctx, lens, hq, hkv, page, seed=len(ctx), qstd=qstd, tail=3)
    call, out, lse = _run(pkg, c)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    _check(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("hint,splits", [(0, 2), (1, 32), (4, 5), (8, 3), (12, 32), (16, 8), (99, 1)])
def test_every_tile_and_split(pkg, hint, splits):
    c = _case([700, 1300, 64], [9, 5, 12], 32, 8, 16, seed=5, qstd=3.0)
    call, out, lse = _run(pkg, c, hint, splits)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    _check(c, out, lse)


BOTH = pytest.mark.parametrize("hint", [2, 8, 12, 16])  # both kernels: 8 (or 16), 32, 48, 64 rows


@pytest.mark.gpu
@BOTH
def test_rising_maxima_and_far_scales(pkg, hint):
    """Scores that grow along the context (every tile moves the running maximum), and
    group scales at both ends of e4m3."""
    c = _case([900], [3], 4, 1, 16, seed=2, qstd=4.0)
    pages = c["table"][0].tolist()
    for i, p in enumerate(pages):
        c["cache"][p, 0, 0, 2048:2112] = torch.tensor(0.02 * 1.12 ** i / c["gk"]).clamp(max=448).to(
            torch.float8_e4m3fn).view(torch.uint8)
    c["cache"][pages[-1], 0, 0, 2048 + 16:2112] = 0x7f      # (900 = 56 * 16 + 4)
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    _check(c, out, lse)
    c = _case([200], [2], 4, 2, 16, seed=3, gk=1.0, gv=1.0)
    lo = torch.randint(0, 2, c["cache"][..., 2112:].shape, generator=torch.Generator().manual_seed(1))
    c["cache"][..., 2112:] = torch.where(lo > 0, 1, 0x7e).to(torch.uint8)     # 2^-9 and 448
    c["cache"][int(c["table"][0, 12]), :, 0, 2112:].view(2, 4, 16)[:, :, 8:] = 0x7f
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    _check(c, out, lse)


@pytest.mark.gpu
@BOTH
def test_query_rows_of_very_different_size(pkg, hint):
    c = _case([300], [4], 4, 2, 16, seed=4)
    for i, f in enumerate((1e-20, 1e-3, 30.0, 0.0)):
        c["q"][i] *= f
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    _check(c, out, lse)


@pytest.mark.gpu
@BOTH
def test_nan_query_stays_in_its_row(pkg, hint):
    c = _case([200, 40], [3, 2], 8, 2, 16, seed=6)
    c["q"][1, 3, 7] = float("nan")
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    assert bool(out[1, 3].isnan().all())
    c["q"][1, 3] = 0
    o, l, _, _ = _reference(c)
    out[1, 3], lse[1, 3] = torch.tensor(o[1, 3]).bfloat16(), float(l[1, 3])
    _check(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("hint", [1, 20])
def test_many_short_requests(pkg, hint):
    """The largest batch, empty requests among it: more items to a CTA than it keeps at hand."""
    B = 1024
    c = _case([(7 * i) % 25 for i in range(B)], [(5 * i) % 3 for i in range(B)], 16, 16, 16, seed=11)
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    _check(c, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("hint", [1, 20])
def test_more_than_2_to_20_tiles(pkg, hint):
    """Contexts of 2^21 tokens whose page tables repeat two pages: every key counts 4096 times."""
    B, H, R = 8, 8, 4096
    c = _case([512], [1], H, H, 256, seed=12)
    short, one = c["table"], {k: c[k] for k in ("q", "k_new", "v_new")}
    for k in one:
        c[k] = one[k].repeat(B, 1, 1)
    c.update(table=short.repeat(B, R), ctx=torch.full((B,), 512 * R, dtype=torch.int32),
             cu=torch.arange(B + 1, dtype=torch.int32), M=B)
    call, out, lse = _run(pkg, c, hint, 32)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    K, V = O.kv4_values(c["cache"].numpy(), c["gk"], c["gv"])
    for h in range(H):
        pages = short[0].numpy()
        k = np.concatenate([K[pages, :, h].reshape(-1, 128), one["k_new"][:, h].double().numpy()])
        v = np.concatenate([V[pages, :, h].reshape(-1, 128), one["v_new"][:, h].double().numpy()])
        x = c["scale"] * k @ one["q"][0, h].double().numpy()
        w = np.exp(x - x.max()) * np.where(np.arange(513) < 512, R, 1)
        o = w @ v / w.sum()
        # sums over 2^21 keys in fp32: a CTA's part holds at most ceil(2^20 / 304) tiles, 2^18.8 keys,
        # of which a thread adds one per tile (2^11.8) and the products eight steps (2^14.8)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2.0 ** 14.8 * 2.0 ** -23) * np.abs(v).max()
        assert (np.abs(out[:, h].double().cpu().numpy() - o) <= tol).all()
        assert (np.abs(lse[:, h].double().cpu().numpy() - x.max() - np.log(w.sum())) <= 2.0 ** -10).all()


@pytest.mark.gpu
@BOTH
def test_long_context_is_split(pkg, hint):
    c = _case([20011], [2], 8, 2, 64, seed=7)
    for splits in (2, 32):
        call, out, lse = _run(pkg, c, hint, splits)
        call()
        torch.cuda.synchronize()
        assert pkg.read_device_error() == 0
        _check(c, out, lse)


@pytest.mark.gpu
@BOTH
def test_bad_page_and_row_overflow(pkg, hint):
    c = _case([200, 100], [3, 2], 8, 2, 16, seed=8)
    for bad in (-5, c["cache"].shape[0]):
        keep = c["table"].clone()
        c["table"][0, 3] = bad
        call, out, lse = _run(pkg, c, hint)
        call()
        assert pkg.read_device_error() == 0x10
        c["table"] = keep
        o, l, _, _ = _reference(c)       # the other request is as ever
        out[:3], lse[:3] = torch.tensor(o[:3]).bfloat16().cuda(), torch.tensor(l[:3]).float().cuda()
        _check(c, out, lse)
    d = dict(c)
    for k in ("q", "k_new", "v_new"):
        d[k] = c[k][:4]
    call, out, lse = _run(pkg, d, hint)
    call()
    assert pkg.read_device_error() == 0x1
    assert bool((out == 5.0).all())


@pytest.mark.gpu
@BOTH
def test_negative_lengths_are_refused(pkg, hint):
    for key, value in (("cu", [0, 4, 3, 5]), ("cu", [2, 0, 3, 5]), ("ctx", [20, -1, 30]),
                       ("ctx", [20, 2 ** 31 - 1, 30])):
        c = _case([20, 40, 30], [1, 2, 2], 4, 2, 16, seed=13)
        c[key] = torch.tensor(value, dtype=torch.int32)
        call, out, lse = _run(pkg, c, hint)
        call()
        assert pkg.read_device_error() == 0x10
        assert bool((out == 5.0).all()) and bool((lse == 5.0).all())


@pytest.mark.gpu
def test_graph_streams_and_repeatability(pkg):
    c = _case([900, 300, 2100], [5, 9, 1], 32, 8, 16, seed=9)
    call, out, lse = _run(pkg, c)
    call()
    torch.cuda.synchronize()
    first, l1 = out.clone(), lse.clone()
    _check(c, out, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.fill_(0)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, l1)
    # two calls at once, each with its own workspace
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [_run(pkg, c, stream=s) for s in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for r in runs:
            r[0]()
    torch.cuda.synchronize()
    for _, o, l in runs:
        assert torch.equal(o, first) and torch.equal(l, l1)
    assert pkg.read_device_error() == 0
