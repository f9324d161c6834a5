"""The 4-bit paged KV cache (dspark_kv4_store / _load, dspark_compact_kv4): codes, scales
and bytes bit for bit against the oracle, and refusals.  The rule is fp32 arithmetic with
IEEE division on both sides, so there is no tolerance."""
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


# ------------------------------------------------------------------ oracle pins (CPU)
def test_oracle_e4m3_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, O._E4M3)


def test_oracle_rule_by_hand():
    x = np.zeros(128, np.float32)
    x[:3] = [7.0, -3.4, 0.5]                   # amax 7, g 1: scale 1; ties to even
    x[32:35] = [7.1, 7.1, -7.1]                # t = 1.0143: the next e4m3 is 1.125
    c, s, v = O.kv4_quantise(x, 1.0)
    assert list(c[:4]) == [15, 5, 8, 8] and O.e4m3_value(s[0]) == 1.0
    assert O.e4m3_value(s[1]) == 1.125 and list(c[32:35]) == [14, 14, 2]
    assert list(v[32:35]) == [6.75, 6.75, -6.75] and s[2] == 0 and c[64] == 8
    big, bs, bv = O.kv4_quantise(np.full(128, 1e6, np.float32), 1.0)
    assert bv[0] == 7 * 448 and big[0] == 15
    x[0], x[1] = np.nan, np.inf
    c, s, v = O.kv4_quantise(x, 1.0)
    assert v[0] == 0 and v[1] == 7 * 448


def test_oracle_half_step_and_round_trip():
    rng = np.random.default_rng(0)
    k, v = (rng.normal(size=(40, 2, 128)).astype(np.float32) * s for s in (3, 0.1))
    cache = rng.integers(0, 256, size=(6, 2, 1, O.KV4_BLOCK_BYTES), dtype=np.uint8)
    cache &= 0x77                              # no NaN scales
    table = np.array([[3, 0, 5], [1, 4, 2]])
    cu, pos0 = np.array([0, 27, 40]), np.array([7, 30])
    new = O.kv4_store(k, v, cu, pos0, table, cache, 0.25, 0.01)
    K, V = O.kv4_values(new, 0.25, 0.01)
    K0, V0 = O.kv4_values(cache, 0.25, 0.01)
    seen = np.zeros(K.shape[:2], bool)
    for r in range(2):
        for i in range(cu[r + 1] - cu[r]):
            p, t = divmod(pos0[r] + i, 16)
            for X, x, g in ((K, k, 0.25), (V, v, 0.01)):
                _, s, val = O.kv4_quantise(x[cu[r] + i], g)
                np.testing.assert_allclose(X[table[r][p], t], val, rtol=1e-6)
                half = 0.5 * O._E4M3[s].repeat(32, axis=-1) * g
                assert np.all(np.abs(val - x[cu[r] + i]) <= half * (1 + 2.0 ** -20))
            seen[table[r][p], t] = True
    assert np.array_equal(K[~seen], K0[~seen]) and np.array_equal(V[~seen], V0[~seen])


# ------------------------------------------------------------------ refusals (CPU)
def test_host_refusals(pkg):
    lib, f, off = pkg.load(), ctypes.c_void_p(4096), ctypes.c_void_p(4100)

    def store(k=f, ks=256, dt=1, cu=f, pos=f, B=2, rows=8, hkv=2, page=16, tab=f, gk=1.0, gv=1.0,
              c=f):
        return lib.dspark_kv4_store(k, ks, f, 256, dt, cu, pos, B, rows, hkv, page, tab, 4, 9, gk,
                                    gv, c, None)

    def load(c=f, pos=f, page=16, gk=1.0, dt=1, k=f, B=2, rows=8):
        return lib.dspark_kv4_load(c, f, pos, B, rows, 2, page, f, 4, 9, gk, 1.0, dt, k, f, None)

    for bad in (dict(k=None), dict(cu=None), dict(pos=None), dict(tab=None), dict(c=None),
                dict(k=off), dict(c=off), dict(ks=248), dict(ks=260), dict(dt=3), dict(B=0),
                dict(B=1025), dict(rows=0), dict(hkv=0), dict(gk=0.0), dict(gk=-1.0),
                dict(gv=float("nan")), dict(gv=float("inf"))):
        assert store(**bad) == -1, bad
    assert store(page=8) == -2 and store(page=48) == -2 and store(rows=1 << 30, hkv=2) == -2
    for bad in (dict(c=None), dict(pos=None), dict(gk=0.0), dict(dt=9), dict(k=off), dict(rows=0)):
        assert load(**bad) == -1, bad
    assert load(page=24) == -2

    def compact(rows=8, gamma=4, c=f, ws=f, n=1 << 20, kn=f):
        return lib.dspark_compact_kv4(kn, f, 2, rows, f, f, f, f, 2, gamma, 16, 4, 9, f, f, f, f, f,
                                      c, 1.0, 1.0, f, f, ws, n, None)

    assert compact(gamma=33) == -1 and compact(c=None) == -1 and compact(kn=off) == -1
    assert compact(ws=ctypes.c_void_p(4112)) == -1 and compact(ws=None) == -1


def test_binding_refusals(pkg):
    with pytest.raises(ValueError):
        pkg.kv4_cache(4, 2, 24, device="cpu")
    c = pkg.kv4_cache(4, 2, 32, device="cpu")
    assert c.shape == (4, 2, 2, pkg.KV4_BLOCK_BYTES) == (4, 2, 2, O.KV4_BLOCK_BYTES)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(3, 2, 128)
    with pytest.raises(ValueError):      # host tensors
        pkg.kv4_store(k, k, i(3), i(2), i(2, 4), c)
    with pytest.raises(ValueError):      # a table of other requests
        pkg.kv4_store(k, k, i(3), i(2), i(3, 4), c)
    with pytest.raises(ValueError):
        pkg.kv4_load(c[..., :-1], i(3), i(2), i(2, 4), k, k)


# ------------------------------------------------------------------ parity (GPU)
def _case(lens, pos0, hkv, page, dtype, seed, extra_pages=3):
    g = torch.Generator().manual_seed(seed)
    rows = sum(lens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k = (2 * torch.randn(rows, hkv, 128, generator=g)).to(dt)
    v = (0.1 * torch.randn(rows, hkv, 128, generator=g)).to(dt)
    need = [-(-(p + n) // page) for p, n in zip(pos0, lens)]
    n_pages = sum(need) + extra_pages
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    cache = torch.randint(0, 256, (n_pages, hkv, page // 16, O.KV4_BLOCK_BYTES), generator=g,
                          dtype=torch.uint8)
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    return k, v, cu, torch.tensor(pos0, dtype=torch.int32), table, cache


LENS = [
    ([1], [0], 1, 16, "bf16"),
    ([1, 9, 3, 0, 5], [15, 30, 16, 7, 0], 2, 16, "bf16"),
    ([40, 1, 70, 17], [3, 64, 0, 111], 3, 64, "f32"),
    ([0, 0, 33, 0], [5, 6, 8, 1], 8, 32, "bf16"),
    ([300, 0, 211], [1, 0, 250], 8, 16, "bf16"),
    # many rows: 16 rows and several heads to a CTA, among them a window of many requests
    ([1900, 0, 611], [1, 0, 250], 4, 16, "bf16"),
    ([(7 * i) % 6 for i in range(500)], [(11 * i) % 70 for i in range(500)], 9, 16, "bf16"),
    ([0] * 40 + [1024] + [0] * 40 + [3] * 9, [5] * 90, 10, 32, "f32"),
    ([1] * 70, list(range(70)), 4, 16, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,pos0,hkv,page,dtype", LENS)
@pytest.mark.parametrize("tail", [0, 5])
def test_store_and_load(pkg, lens, pos0, hkv, page, dtype, tail):
    k, v, cu, p0, table, cache = _case(lens, pos0, hkv, page, dtype, 3)
    gk, gv = 0.0625, 0.0173
    dev = cache.cuda()
    rows = k.shape[0]
    fused = torch.cat([k.flatten(1), v.flatten(1)], 1).cuda()
    fused = torch.cat([fused, fused.new_full((tail, fused.shape[1]), float("nan"))])  # rows past M
    kd, vd = (x.unflatten(1, (-1, 128)) for x in fused.split(hkv * 128, 1))
    pkg.kv4_store(kd, vd, cu.cuda(), p0.cuda(), table.cuda(), dev, gk, gv)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    ref = O.kv4_store(k.float().numpy(), v.float().numpy(), cu.numpy(), p0.numpy(), table.numpy(),
                      cache.numpy(), gk, gv)
    assert np.array_equal(dev.cpu().numpy(), ref)
    for dt in (torch.float32, torch.bfloat16):
        ko = torch.full((rows + tail, hkv, 128), 9.0, dtype=dt, device="cuda")
        vo = torch.full_like(ko, 9.0)
        pkg.kv4_load(dev, cu.cuda(), p0.cuda(), table.cuda(), ko, vo, gk, gv)
        torch.cuda.synchronize()
        assert pkg.read_device_error() == 0
        for got, x, g in ((ko, k, gk), (vo, v, gv)):
            want = torch.tensor(O.kv4_quantise(x.float().numpy(), g)[2]).float().to(dt)
            assert torch.equal(got[:rows].cpu(), want)
            assert bool((got[rows:] == 9.0).all())


@pytest.mark.gpu
def test_extreme_values(pkg):
    k, v, cu, p0, table, cache = _case([6], [12], 2, 16, "f32", 1)
    k[0, 0, 3], k[0, 0, 4] = float("nan"), 2.0
    k[1, 1, 40] = float("inf")
    k[2] = 0
    k[3] *= 1e30
    k[4] *= 1e-30
    v[0, 0] = -float("inf")
    v[1, 0, 5:40] = float("nan")
    v[2] = 1e-45
    dev = cache.cuda()
    pkg.kv4_store(k.cuda(), v.cuda(), cu.cuda(), p0.cuda(), table.cuda(), dev, 0.5, 0.5)
    torch.cuda.synchronize()
    ref = O.kv4_store(k.numpy(), v.numpy(), cu.numpy(), p0.numpy(), table.numpy(), cache.numpy(),
                      0.5, 0.5)
    assert np.array_equal(dev.cpu().numpy(), ref)


@pytest.mark.gpu
def test_bad_pages_and_row_overflow_change_nothing_else(pkg):
    k, v, cu, p0, table, cache = _case([20, 4], [10, 3], 2, 16, "bf16", 2)
    for r, slot, page in ((0, 1, -1), (1, 0, cache.shape[0])):
        tab = table.clone()
        tab[r, slot] = page
        dev = cache.cuda()
        pkg.read_device_error()
        pkg.kv4_store(k.cuda(), v.cuda(), cu.cuda(), p0.cuda(), tab.cuda(), dev, 1.0, 1.0)
        assert pkg.read_device_error() == 0x10
        # the other blocks are stored
        good = O.kv4_store(k.float().numpy(), v.float().numpy(), cu.numpy(), p0.numpy(),
                           table.numpy(), cache.numpy(), 1.0, 1.0)
        got = dev.cpu().numpy()
        bad = int(table[r, slot])
        assert np.array_equal(np.delete(got, bad, 0), np.delete(good, bad, 0))
        assert np.array_equal(got[bad], cache.numpy()[bad])
        out = [torch.full((24, 2, 128), 9.0, device="cuda") for _ in range(2)]
        pkg.kv4_load(dev, cu.cuda(), p0.cuda(), tab.cuda(), *out, 1.0, 1.0)
        assert pkg.read_device_error() == 0x10
    far = torch.tensor([10, 1000], dtype=torch.int32)      # past the page table's row
    dev = cache.cuda()
    pkg.kv4_store(k.cuda(), v.cuda(), cu.cuda(), far.cuda(), table.cuda(), dev, 1.0, 1.0)
    assert pkg.read_device_error() == 0x10
    dev = cache.cuda()                                     # cu_seqlens past the rows
    pkg.kv4_store(k[:20].cuda(), v[:20].cuda(), cu.cuda(), p0.cuda(), table.cuda(), dev, 1.0, 1.0)
    assert pkg.read_device_error() == 0x1
    assert torch.equal(dev.cpu(), cache)


@pytest.mark.gpu
def test_store_in_a_graph_on_another_stream(pkg):
    k, v, cu, p0, table, cache = _case([9, 2, 31], [4, 15, 60], 8, 16, "bf16", 4)
    dev = cache.cuda()
    args = [t.cuda() for t in (k, v, cu, p0, table)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.kv4_store(*args, dev, 0.1, 0.2)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    ref = O.kv4_store(k.float().numpy(), v.float().numpy(), cu.numpy(), p0.numpy(), table.numpy(),
                      cache.numpy(), 0.1, 0.2)
    assert np.array_equal(dev.cpu().numpy(), ref)
    other = cache.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pkg.kv4_store(*args, other, 0.1, 0.2, stream=s)
    s.synchronize()
    assert torch.equal(other, dev)


@pytest.mark.gpu
@pytest.mark.parametrize("B,gamma,hkv,page", [(1, 1, 1, 16), (7, 6, 2, 16), (40, 16, 8, 64), (200, 6, 18, 16)])
def test_compact_kv4(pkg, B, gamma, hkv, page):
    rng = np.random.default_rng(B)
    ctx = rng.integers(0, 3 * page, size=B)
    acc = rng.integers(0, gamma + 1, size=B)
    n = np.minimum(acc + 1 + rng.integers(0, 3, size=B), gamma + 1)
    have = -(-ctx // page)
    max_pages = int(max(-(-(ctx + acc + 1) // page))) + 1
    n_pages = int(have.sum()) + 2 * B + 2
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.zeros((B, max_pages), np.int32)
    at = 0
    for r in range(B):
        table[r, :have[r]] = perm[at:at + have[r]]
        at += have[r]
    free = perm[at:].copy()
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    rows = int(cu[-1]) + 3
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(rows, hkv, 128, generator=g).bfloat16() for _ in range(2))
    cache = torch.randint(0, 256, (n_pages, hkv, page // 16, O.KV4_BLOCK_BYTES), generator=g,
                          dtype=torch.uint8)
    tok = rng.integers(0, 999, size=(B, gamma)).astype(np.int32)
    out_tok = rng.integers(0, 999, size=B).astype(np.int32)
    d = {k_: torch.tensor(np.asarray(x, dtype=np.int32)).cuda() for k_, x in dict(
        cu=cu, acc=acc, out=out_tok, tok=tok, table=table, ctx=ctx, anchor=np.zeros(B), free=free,
        top=[len(free)], com=np.zeros((B, gamma + 1)), ncom=np.zeros(B)).items()}
    dev = cache.cuda()
    ws = torch.empty(pkg.compact_workspace_size(B), dtype=torch.uint8, device="cuda")
    pkg.compact_kv4(k.cuda(), v.cuda(), d["cu"], d["acc"], d["out"], d["tok"], d["table"], d["ctx"],
                    d["anchor"], d["free"], d["top"], dev, d["com"], d["ncom"], ws, 0.5, 0.25)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    z = np.zeros((n_pages, page, 1, 16), np.float32)       # the page bookkeeping alone
    ref = O.compact(np.zeros((rows, 1, 16), np.float32), np.zeros((rows, 1, 16), np.float32), cu, acc,
                    out_tok, tok, page, table, ctx.astype(np.int32), np.zeros(B, np.int32), free,
                    len(free), z, z)
    assert np.array_equal(d["table"].cpu().numpy(), ref.page_table)
    assert np.array_equal(d["ctx"].cpu().numpy(), ref.ctx_len)
    assert int(d["top"]) == ref.free_top and np.array_equal(d["com"].cpu().numpy(), ref.committed)
    want = O.kv4_store(k.float().numpy(), v.float().numpy(), cu, ctx, ref.page_table, cache.numpy(),
                       0.5, 0.25, n_keep=acc + 1)
    assert np.array_equal(dev.cpu().numpy(), want)
    # no free page: nothing changes
    d["top"].zero_()
    d["ctx"].copy_(torch.tensor(np.full(B, page, np.int32)))
    d["table"][:, 0] = 0
    before = dev.clone()
    pkg.compact_kv4(k.cuda(), v.cuda(), d["cu"], d["acc"], d["out"], d["tok"], d["table"], d["ctx"],
                    d["anchor"], d["free"], d["top"], dev, d["com"], d["ncom"], ws, 0.5, 0.25)
    assert pkg.read_device_error() == 0x2
    assert torch.equal(dev, before)
