"""Verify attention of drafted trees (dspark_verify_attn_tree) against the softmax of its definition
in fp64, and its refusals.

Tolerance, from the arithmetic (S = max over a row's keys of scale * sum |q k|, A = the weighted sum of
|v|, n the row's keys):
  * a score is a sum of 128 products, exact in fp32, accumulated in fp32 (each step off by at most
    2^-23): 128 * 2^-23 S; its scaling and the exponential's argument add 8 * 2^-23 S, the exponential
    2^-21.  Together es; a weight is off by 2 es relative (its own and the normaliser's).
  * probabilities are rounded to bf16: 2^-8 each; one below 2^-126 of the largest may be dropped.
  * sums over n keys in fp32: n 2^-23, and a merge of split pieces 64 * 2^-23.
  * the output's own rounding to bf16: 2^-8 of the value.
The lse is off by es and the sums."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O
from tests.test_tree import forest


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import speculative_decoding_verification_dspark_gb300 as p
    return p


def check(out, lse, want, n):
    o, l, S, A = want
    es = (136 * S + 4) * 2.0 ** -23
    rel = 2 * es + (n + 64) * 2.0 ** -23
    tol = A * (rel[..., None] + 2.0 ** -8) + np.abs(o) * 2.0 ** -8 + 1e-30
    np.testing.assert_array_equal(np.isnan(out), np.isnan(o))
    bad = np.abs(out - o) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.nanmax(np.abs(out - o) / tol))
    empty = l == -np.inf
    np.testing.assert_array_equal(lse == -np.inf, empty)
    some = ~empty & ~np.isnan(l)
    d, most = np.abs(lse[some] - l[some]), (es + (n + 64) * 2.0 ** -23 + np.abs(l) * 2.0 ** -23)[some]
    assert (d <= most).all(), (d / most).max()


class Case:
    def __init__(self, sizes, ctx, Hq, Hkv, page, seed=0, kind="mixed", pad=3, words=None):
        rng = np.random.default_rng(seed)
        self.cu, self.parent = forest(sizes, rng, kind)
        self.B, self.live, self.n_max = len(sizes), int(self.cu[-1]), max(max(sizes), 1)
        self.ctx = np.array(ctx, np.int32)
        need = -(-self.ctx // page)
        n_pages = int(need.sum()) + 2
        perm = rng.permutation(n_pages).astype(np.int32)
        self.table = np.zeros((self.B, max(int(need.max()), 1)), np.int32)
        at = 0
        for r in range(self.B):
            self.table[r, :need[r]] = perm[at:at + need[r]]
            at += need[r]
        g = torch.Generator().manual_seed(seed)
        rows = self.live + pad

        def rand(*s):
            return torch.randn(*s, generator=g).bfloat16()

        self.q, self.kn, self.vn = 1.5 * rand(rows, Hq, 128), rand(rows, Hkv, 128), rand(rows, Hkv, 128)
        self.kc, self.vc = rand(n_pages, page, Hkv, 128), rand(n_pages, page, Hkv, 128)
        self.words = words or -(-self.n_max // 64)
        self.mask = np.zeros((rows, self.words), np.uint64)
        self.mask[:self.live] = O.tree_masks(self.parent, self.cu, self.ctx, max(self.words, -(-self.n_max // 64)))[0][:, :self.words]
        self.scale, self.Hq, self.Hkv, self.rows, self.page = 128 ** -0.5, Hq, Hkv, rows, page

    def run(self, pkg, hint=None, splits=32, stream=None):
        hint = self.n_max if hint is None else hint
        dev = {k: getattr(self, k).cuda() for k in ("q", "kn", "vn", "kc", "vc")}
        i = {k: torch.tensor(getattr(self, k), device="cuda") for k in ("table", "ctx", "cu")}
        mask = torch.tensor(self.mask.view(np.int64), device="cuda")
        out = torch.full((self.rows, self.Hq, 128), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.rows, self.Hq), 77.0, device="cuda")
        ws = torch.empty(pkg.verify_attn_tree_workspace_size(self.B, self.rows, self.Hq, self.Hkv, splits, hint),
                         dtype=torch.uint8, device="cuda")
        ws.fill_(0xA5)
        pkg.verify_attn_tree(dev["q"], dev["kn"], dev["vn"], dev["kc"], dev["vc"], i["table"], i["ctx"], i["cu"],
                             mask, self.scale, splits, out, lse, ws, stream, max_block_rows=hint)
        torch.cuda.synchronize()
        self.err = pkg.read_device_error()
        return out, lse

    def want(self):
        f = lambda t: t.float().numpy()  # noqa: E731
        return O.verify_attention_tree(f(self.q)[:self.live], f(self.kn)[:self.live], f(self.vn)[:self.live],
                                       f(self.kc), f(self.vc), self.table, self.ctx, self.cu,
                                       self.mask[:self.live], self.scale)

    def verify(self, pkg, **kw):
        out, lse = self.run(pkg, **kw)
        assert self.err == 0, hex(self.err)
        o, l = out.float().cpu().numpy(), lse.cpu().numpy()
        check(o[:self.live], l[:self.live], self.want(), int(self.ctx.max()) + self.n_max)
        assert (o[self.live:] == 77).all() and (l[self.live:] == 77).all()
        return out, lse


# ------------------------------------------------------------------ refusals (CPU)
def test_host_refusals(pkg):
    lib, f, off = pkg.load(), ctypes.c_void_p(4096), ctypes.c_void_p(4104)

    def call(q=f, kc=f, tab=f, ctx=f, cu=f, mask=f, words=1, B=2, rows=8, hq=8, hkv=2, page=16, scale=0.1,
             splits=8, hint=4, out=f, lse=f, ws=f, n=1 << 40, pages=9):
        return lib.dspark_verify_attn_tree(q, f, f, kc, f, pages, tab, 4, ctx, cu, mask, words, B, rows, hq, hkv,
                                           page, ctypes.c_float(scale), splits, hint, out, lse, ws, n, None)

    for bad in (dict(q=None), dict(kc=None), dict(tab=None), dict(ctx=None), dict(cu=None), dict(mask=None),
                dict(out=None), dict(lse=None), dict(ws=None), dict(q=off), dict(kc=off), dict(out=off),
                dict(ws=off), dict(words=0), dict(words=9), dict(B=0), dict(B=1025), dict(rows=0),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(splits=0), dict(splits=33), dict(pages=0)):
        assert call(**bad) == -1, bad
    for bad in (dict(hq=9), dict(hq=258), dict(hkv=0), dict(page=8), dict(page=40)):
        assert call(**bad) == -2, bad
    size = lib.dspark_verify_attn_tree_workspace_size
    assert size(2, 8, 9, 2, 8, 4) == 0 and size(0, 8, 8, 2, 8, 4) == 0 and size(2, 0, 8, 2, 8, 1) == 0
    assert size(32, 512, 32, 8, 8, 0) > 0


def test_binding_refusals(pkg):
    bf, i32 = torch.bfloat16, torch.int32
    q, kn = torch.zeros(8, 8, 128, dtype=bf), torch.zeros(8, 2, 128, dtype=bf)
    kc, tab = torch.zeros(4, 16, 2, 128, dtype=bf), torch.zeros(2, 4, dtype=i32)
    ctx, cu, mask = torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(8, 1, dtype=torch.int64)
    ws = torch.zeros(64, dtype=torch.uint8)
    args = [q, kn, kn, kc, kc, tab, ctx, cu, mask, 0.1, 8, q, torch.zeros(8, 8), ws]
    with pytest.raises(ValueError, match="current CUDA device"):
        pkg.verify_attn_tree(*args)
    for at, bad, match in ((0, q.float(), "q"), (3, kc[..., :64], "k_cache"), (8, mask[:, 0], "row_mask"),
                           (5, tab[:1], "page_table"), (1, kn[:7], "k_new|current")):
        a = list(args)
        a[at] = bad
        with pytest.raises(ValueError, match=match):
            pkg.verify_attn_tree(*a)


# ------------------------------------------------------------------ on the GPU
@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (4, 4), (7, 1), (40, 8), (33, 1), (128, 1)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_heads_and_pages(pkg, Hq, Hkv, page):
    Case([5, 1, 20], [130, 0, 517], Hq, Hkv, page, seed=Hq + page).verify(pkg)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 1000])
def test_context_lengths(pkg, ctx):
    Case([3, 33], [ctx, max(0, ctx - 1)], 8, 2, 16, seed=ctx).verify(pkg)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 256, 300, 512])
@pytest.mark.parametrize("G", [1, 4])
def test_tree_sizes(pkg, n, G):
    Case([n], [77], G, 1, 16, seed=n).verify(pkg)


@pytest.mark.gpu
@pytest.mark.parametrize("hint", [0, 1, 8, 40, 1000])
def test_any_hint(pkg, hint):
    a = Case([1, 70, 0, 40], [300, 20, 9, 0], 16, 4, 32, seed=5)
    a.verify(pkg, hint=hint)


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [1, 2, 7, 32])
@pytest.mark.parametrize("sizes,ctx", [([9], [6000]), ([40, 3], [3000, 9000])])
def test_splits(pkg, splits, sizes, ctx):
    Case(sizes, ctx, 8, 2, 64, seed=splits).verify(pkg, splits=splits)


@pytest.mark.gpu
def test_many_requests(pkg):
    rng = np.random.default_rng(2)
    Case(rng.integers(0, 12, 300), rng.integers(0, 400, 300), 8, 2, 16).verify(pkg)


@pytest.mark.gpu
def test_free_masks(pkg):
    """Masks that no tree gives: rows that see nothing, not themselves, rows behind them, all."""
    c = Case([70, 20], [0, 40], 8, 2, 16, words=2)
    rng = np.random.default_rng(0)
    c.mask[:] = rng.integers(0, 1 << 63, c.mask.shape, dtype=np.uint64) * np.uint64(2)
    c.mask[3] = 0                                   # context 0: sees no key at all
    c.mask[10] = ~np.uint64(0)
    c.mask[75] = 0                                  # its context alone
    out, lse = c.verify(pkg)
    assert (out[3] == 0).all() and (lse[3] == -np.inf).all()


@pytest.mark.gpu
def test_rows_past_the_words_are_unseen(pkg):
    c = Case([100], [5], 8, 2, 16, kind="chain", words=1)
    c.verify(pkg)


@pytest.mark.gpu
@pytest.mark.parametrize("val", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("what", ["kn", "vn"])
def test_unseen_block_rows_have_no_effect(pkg, val, what):
    """Row 2 of the block holds `val`; rows that do not see it come out as without it."""
    c = Case([40], [50], 8, 2, 16, kind="mixed", seed=4)
    clean = c.run(pkg)[0].clone()
    getattr(c, what)[2, :, 5] = val
    out = c.run(pkg)[0]
    sees = (c.mask[:40, 0] >> np.uint64(2)) & np.uint64(1) > 0
    assert 0 < sees.sum() < 39
    assert torch.equal(out[:40][~sees], clean[:40][~sees])
    got = out[:40][sees].float()
    if what == "vn":
        assert not torch.isfinite(got[..., 5]).any()
        other = [d for d in range(128) if d != 5]
        assert torch.equal(got[..., other], clean[:40][sees][..., other].float())
    elif val != val:
        assert torch.isnan(got).all()


@pytest.mark.gpu
def test_stale_slots_and_padding_have_no_effect(pkg):
    """Slots of the last page past the context, other pages, and rows outside the segments hold NaN."""
    c = Case([5, 33], [19, 130], 8, 2, 16, seed=6, pad=20)
    clean = c.run(pkg)[0].clone()
    for t in (c.kc, c.vc):
        keep = t.clone()
        t[:] = float("nan")
        for r in range(2):
            for pos in range(c.ctx[r]):
                pg = c.table[r, pos // 16]
                t[pg, pos % 16] = keep[pg, pos % 16]
    for t in (c.q, c.kn, c.vn):
        t[c.live:] = float("nan")
    out = c.run(pkg)[0]
    assert c.err == 0 and torch.equal(out, clean)


@pytest.mark.gpu
def test_other_requests_rows_have_no_effect(pkg):
    c = Case([20, 20], [30, 30], 8, 2, 16, seed=7)
    clean = c.run(pkg)[0].clone()
    for t in (c.kn, c.vn):
        t[20:40] = float("nan")
    out = c.run(pkg)[0]
    assert torch.equal(out[:20], clean[:20]) and torch.isnan(out[20:40].float()).any()


@pytest.mark.gpu
def test_infinite_scores(pkg):
    """A key whose score is -inf weighs nothing; a row with no other sees none."""
    c = Case([2], [0], 1, 1, 16, kind="chain")
    c.q[:] = 1.0
    c.kn[0] = 0
    c.kn[0, 0, 0] = -float("inf")
    out, lse = c.run(pkg)
    assert (out[0] == 0).all() and lse[0, 0] == -np.inf
    assert torch.equal(out[1], c.vn[1].cuda())


@pytest.mark.gpu
def test_bad_input(pkg):
    def fresh():
        return Case([3, 4], [20, 30], 8, 2, 16)
    c = fresh()
    c.ctx[1] = -1
    out, _ = c.run(pkg)
    assert c.err == 0x10 and (out == 77).all()
    c = fresh()
    c.cu = np.array([0, 5, 4], np.int32)
    out, _ = c.run(pkg)
    assert c.err == 0x10 and (out == 77).all()
    c = fresh()
    c.cu = np.array([0, 3, 99], np.int32)
    out, _ = c.run(pkg)
    assert c.err == 0x1 and (out == 77).all()
    c = fresh()
    c.table[1, 1] = 1 << 20
    clean = fresh().run(pkg)[0]
    out, _ = c.run(pkg)
    assert c.err == 0x10 and torch.equal(out[:3], clean[:3]) and (out[7:] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_shares_of_mixed_batches(pkg, seed):
    """Segments of one and of two query tiles, whose key tiles count differently in the CTAs' shares."""
    rng = np.random.default_rng(seed)
    sizes = [int(rng.choice([0, 1, 31, 32, 33, 64, 65, 130])) for _ in range(9)]
    ctx = [int(rng.choice([0, 1, 127, 128, 700, 2049])) for _ in range(9)]
    Case(sizes, ctx, 4, 1, 32, seed=seed).verify(pkg, splits=int(rng.choice([1, 3, 32])))
