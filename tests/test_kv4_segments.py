"""The 4-bit cache's calls on a part of a larger batch: cu_seqlens that begins past row 0 (a
slice cu[3:] of a batch's), against the oracle, bit for bit, and refused where it begins before."""
import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O
from tests.test_kv4_cache import pkg  # noqa: F401
from tests.test_verify_attn_kv4 import BOTH, _case, _reference, _run

pytestmark = pytest.mark.gpu


def _batch(cu, pos0, hkv, page, seed, tail=3):
    g = torch.Generator().manual_seed(seed)
    rows, B = cu[-1] + tail, len(pos0)
    k, v = (torch.randn(rows, hkv, 128, generator=g).bfloat16() for _ in range(2))
    need = [-(-(p + cu[r + 1] - cu[r]) // page) for r, p in enumerate(pos0)]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    cache = torch.randint(0, 256, (n_pages, hkv, page // 16, O.KV4_BLOCK_BYTES), generator=g,
                          dtype=torch.uint8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return k, v, i32(cu), i32(pos0), table, cache


CUTS = [  # cu, pos0, hkv, page
    ([32, 40], [70], 2, 16),             # rows 10 and 26 would be positions 48 and 64
    ([1, 2], [1], 1, 16),
    ([33, 33, 60, 61], [500, 70, 15], 3, 64),
    ([4000, 5000, 5003], [7000, 9], 4, 16),  # 16 rows and several heads to a CTA
]


@pytest.mark.parametrize("cu,pos0,hkv,page", CUTS)
def test_store_and_load_of_a_part(pkg, cu, pos0, hkv, page):  # noqa: F811
    k, v, cut, p0, table, cache = _batch(cu, pos0, hkv, page, 1)
    dev = cache.cuda()
    pkg.kv4_store(k.cuda(), v.cuda(), cut.cuda(), p0.cuda(), table.cuda(), dev, 0.25, 0.5)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    want = O.kv4_store(k.float().numpy(), v.float().numpy(), cut.numpy(), p0.numpy(), table.numpy(),
                       cache.numpy(), 0.25, 0.5)
    assert np.array_equal(dev.cpu().numpy(), want)
    ko, vo = (torch.full((k.shape[0], hkv, 128), 9.0, device="cuda") for _ in range(2))
    pkg.kv4_load(dev, cut.cuda(), p0.cuda(), table.cuda(), ko, vo, 0.25, 0.5)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    for got, x, g in ((ko, k, 0.25), (vo, v, 0.5)):
        value = torch.tensor(O.kv4_quantise(x.float().numpy(), g)[2]).float()
        assert torch.equal(got[cu[0]:cu[-1]].cpu(), value[cu[0]:cu[-1]])
        assert bool((got[:cu[0]] == 9.0).all()) and bool((got[cu[-1]:] == 9.0).all())


def test_compact_of_a_part(pkg):  # noqa: F811
    """Requests 2 and 3 of a batch: what the whole batch's commit does for them."""
    k, v, cu, ctx, table, cache = _batch([37, 42, 44], [75, 16], 2, 16, 2)
    gamma, B = 4, 2
    acc, tok = [3, 1], torch.arange(B * gamma, dtype=torch.int32).view(B, gamma)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    dev, d_ctx = cache.cuda(), ctx.cuda()
    # request 0 stays in its fifth page (75 + 4 of 80 positions), request 1 takes a second one
    table_d = table.clone().cuda()
    table_d[1, 1] = -1
    free, top = i32([int(table[1, 1])]), i32([1])
    ws = torch.empty(pkg.compact_workspace_size(B), dtype=torch.uint8, device="cuda")
    com, ncom = z(B, gamma + 1), z(B)
    pkg.compact_kv4(k.cuda(), v.cuda(), cu.cuda(), i32(acc), i32([900, 901]), tok.cuda(), table_d,
                    d_ctx, z(B), free, top, dev, com, ncom, ws, 0.25, 0.5)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    assert d_ctx.tolist() == [79, 18] and int(top) == 0 and torch.equal(table_d.cpu(), table)
    want = O.kv4_store(k.float().numpy(), v.float().numpy(), cu.numpy(), ctx.numpy(), table.numpy(),
                       cache.numpy(), 0.25, 0.5, n_keep=[a + 1 for a in acc])
    assert np.array_equal(dev.cpu().numpy(), want)


@BOTH
def test_attention_of_a_part(pkg, hint):  # noqa: F811
    c = _case([200, 40, 300, 129], [5, 2, 4, 9], 8, 2, 16, seed=31)
    o, lse, to, tl = _reference(c)
    for k in ("cu", "ctx", "table"):
        c[k] = c[k][2:]
    call, out, l = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    assert np.all((np.abs(out.double().cpu().numpy() - o) <= to)[7:])
    assert np.all((np.abs(l.double().cpu().numpy() - lse) <= tl)[7:])
    assert bool((out[:7] == 5.0).all()) and bool((l[:7] == 5.0).all())


@BOTH
def test_attention_refuses_a_first_row_below_zero(pkg, hint):  # noqa: F811
    c = _case([20, 40, 30], [1, 2, 2], 4, 2, 16, seed=32)
    for first in (-1, -300):
        c["cu"] = torch.tensor([first, 1, 3, 5], dtype=torch.int32)
        call, out, lse = _run(pkg, c, hint)
        call()
        assert pkg.read_device_error() == 0x10
        assert bool((out == 5.0).all()) and bool((lse == 5.0).all())


@pytest.mark.parametrize("first", [-1, -300])
@pytest.mark.parametrize("last", [9, 5000])   # a row per CTA, and 16
def test_store_and_load_refuse_a_first_row_below_zero(pkg, first, last):  # noqa: F811
    k, v, cu, p0, table, cache = _batch([0, 3, last], [5, 20], 4, 16, 3)
    cu[0] = first
    dev = cache.cuda()
    args = [t.cuda() for t in (cu, p0, table)]
    pkg.kv4_store(k.cuda(), v.cuda(), *args, dev, 0.25, 0.5)
    assert pkg.read_device_error() == 0x10 and torch.equal(dev.cpu(), cache)
    ko, vo = (torch.full(k.shape, 9.0, device="cuda") for _ in range(2))
    pkg.kv4_load(dev, *args, ko, vo, 0.25, 0.5)
    assert pkg.read_device_error() == 0x10 and bool((ko == 9.0).all()) and bool((vo == 9.0).all())


@pytest.mark.parametrize("kv4", [False, True])
def test_compact_refuses_a_first_row_below_zero(pkg, kv4):  # noqa: F811
    gamma, B, page = 4, 2, 16
    k, v, cu, ctx, table, cache = _batch([0, 3, 6], [14, 20], 2, page, 4)
    cu[0] = -1
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    kept = dict(table=table.cuda(), ctx=ctx.cuda(), anchor=z(B), top=z(1) + 5, com=z(B, gamma + 1),
                ncom=z(B))
    if kv4:
        caches = [cache.cuda()]
    else:
        caches = [torch.ones(cache.shape[0], page, 2, 128, dtype=torch.bfloat16, device="cuda")
                  for _ in range(2)]
    before = [t.clone() for t in (*kept.values(), *caches)]
    ws = torch.empty(pkg.compact_workspace_size(B), dtype=torch.uint8, device="cuda")
    free = torch.arange(5, dtype=torch.int32, device="cuda")
    call, scales = (pkg.compact_kv4, (0.25, 0.5)) if kv4 else (pkg.compact, ())
    call(k.cuda(), v.cuda(), cu.cuda(), z(B) + 1, z(B), z(B, gamma), kept["table"], kept["ctx"],
         kept["anchor"], free, kept["top"], *caches, kept["com"], kept["ncom"], ws, *scales)
    assert pkg.read_device_error() == 0x10
    assert all(torch.equal(a, b) for a, b in zip(before, (*kept.values(), *caches)))


@BOTH
def test_attention_refuses_ends_past_32_bits(pkg, hint):  # noqa: F811
    """Context and rows together: positions of the tiles behind them stay in 32 bits."""
    for ctx, n in ((2 ** 31 - 769, 1), (2 ** 31 - 1000, 300), (2 ** 31 - 258, 300), (2 ** 31 - 2, 2)):
        c = _case([20, 40], [1, n], 2, 1, 16, seed=33)
        c["ctx"][1] = ctx
        call, out, lse = _run(pkg, c, hint)
        call()
        assert pkg.read_device_error() == 0x10
        assert bool((out == 5.0).all()) and bool((lse == 5.0).all())


@BOTH
def test_attention_refuses_rows_that_fall_to_ints_end(pkg, hint):  # noqa: F811
    """The difference of two rows may pass 32 bits and look like a length."""
    c = _case([20, 40, 30], [1, 2, 2], 4, 2, 16, seed=34)
    for cu in ([0, 1, 3, -2 ** 31], [0, 1, 2000, -2 ** 31], [0, 2 ** 31 - 1, -2 ** 31, 5],
               [-2 ** 31, -2 ** 31, -2 ** 31, 0]):
        c["cu"] = torch.tensor(cu, dtype=torch.int32)
        call, out, lse = _run(pkg, c, hint)
        call()
        err = pkg.read_device_error()
        assert err & (0x1 if cu[-1] < 0 else 0x10) and not err & ~0x11
        assert bool((out == 5.0).all()) and bool((lse == 5.0).all())


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("cu_bad", [[0, 3, -2 ** 31], [0, 2000000000, -2 ** 31], [0, 7, 6]])
def test_compact_refuses_rows_that_fall(pkg, cu_bad, kv4):  # noqa: F811
    gamma, B, page = 4, 2, 16
    k, v, cu, ctx, table, cache = _batch([0, 3, 6], [14, 20], 2, page, 4)
    cu[:] = torch.tensor(cu_bad, dtype=torch.int32)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    kept = dict(table=table.cuda(), ctx=ctx.cuda(), anchor=z(B), top=z(1) + 5, com=z(B, gamma + 1),
                ncom=z(B))
    if kv4:
        caches = [cache.cuda()]
    else:
        caches = [torch.ones(cache.shape[0], page, 2, 128, dtype=torch.bfloat16, device="cuda")
                  for _ in range(2)]
    before = [t.clone() for t in (*kept.values(), *caches)]
    ws = torch.empty(pkg.compact_workspace_size(B), dtype=torch.uint8, device="cuda")
    free = torch.arange(5, dtype=torch.int32, device="cuda")
    call, scales = (pkg.compact_kv4, (0.25, 0.5)) if kv4 else (pkg.compact, ())
    call(k.cuda(), v.cuda(), cu.cuda(), z(B) + 1, z(B), z(B, gamma), kept["table"], kept["ctx"],
         kept["anchor"], free, kept["top"], *caches, kept["com"], kept["ncom"], ws, *scales)
    assert pkg.read_device_error() == 0x10
    assert all(torch.equal(a, b) for a, b in zip(before, (*kept.values(), *caches)))
