"""Trees of drafted tokens: masks and positions (tree_pack), the walk (accept_tree) and the commit of
a path (compact with path), whole numbers and bytes bit for bit against the oracle; refusals."""
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


def forest(sizes, rng, kind="mixed"):
    """(cu_seqlens, parents) of trees of these sizes."""
    parent = []
    for n in sizes:
        for i in range(n):
            if i == 0:
                parent.append(-1)
            elif kind == "chain":
                parent.append(i - 1)
            elif kind == "star":
                parent.append(0)
            elif kind == "forest":
                parent.append(int(rng.integers(-1, i)))
            else:
                parent.append(int(rng.integers(max(0, i - 4) if rng.random() < 0.6 else 0, i)))
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32), np.array(parent, np.int32)


# ------------------------------------------------------------------ refusals and pins (CPU)
def test_oracle_by_hand():
    cu, parent = np.array([0, 0, 5], np.int32), np.array([-1, 0, 0, 1, 3], np.int32)
    mask, pos = O.tree_masks(parent, cu, np.array([9, 100], np.int32), 1)
    assert [int(m) for m in mask[:, 0]] == [1, 3, 5, 11, 27] and list(pos) == [100, 101, 101, 102, 103]
    tok, say = np.array([7, 4, 5, 6, 8], np.int32), np.array([4, 6, 0, 9, 1], np.int32)
    path, ptok, n, out = O.accept_tree(tok, parent, say, cu, 4)
    assert list(path[1]) == [0, 1, 3, -1, -1] and list(ptok[1]) == [4, 6, -1, -1]
    assert list(n) == [-1, 2] and list(out) == [-1, 9]
    assert list(O.accept_tree(tok, parent, say, cu, 1)[2]) == [-1, 1]   # no more than gamma drafts


def test_host_refusals(pkg):
    lib, f, off = pkg.load(), ctypes.c_void_p(4096), ctypes.c_void_p(4104)

    def pack(par=f, cu=f, ctx=f, B=2, rows=8, words=1, mask=f, pos=f):
        return lib.dspark_tree_pack(par, cu, ctx, B, rows, words, mask, pos, None)

    for bad in (dict(par=None), dict(cu=None), dict(ctx=None), dict(mask=None), dict(pos=None), dict(B=0),
                dict(B=1025), dict(rows=0), dict(words=0), dict(words=9)):
        assert pack(**bad) == -1, bad

    def accept(tok=f, par=f, say=f, cu=f, B=2, gamma=4, rows=8, path=f, ptok=f, n=f, out=f):
        return lib.dspark_accept_tree(tok, par, say, cu, B, gamma, rows, path, ptok, n, out, None)

    for bad in (dict(tok=None), dict(par=None), dict(say=None), dict(cu=None), dict(path=None),
                dict(ptok=None), dict(n=None), dict(out=None), dict(B=0), dict(gamma=0), dict(gamma=33),
                dict(rows=0)):
        assert accept(**bad) == -1, bad

    def compact(k=f, path=f, gamma=4, kc=f, B=2, ws=f):
        return lib.dspark_compact_path(k, f, 256, 8, f, f, f, f, path, B, gamma, 16, 4, 9, f, f, f, f, f,
                                       kc, f, f, f, ws, 1 << 20, None)

    for bad in (dict(k=None), dict(path=None), dict(gamma=0), dict(kc=off), dict(B=0), dict(ws=off)):
        assert compact(**bad) == -1, bad


def test_binding_refusals(pkg):
    i32 = torch.int32
    par, cu, ctx = torch.zeros(8, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    mask, pos = torch.zeros(8, 1, dtype=torch.int64), torch.zeros(8, dtype=i32)
    with pytest.raises(ValueError, match="current CUDA device"):
        pkg.tree_pack(par, cu, ctx, mask, pos)
    with pytest.raises(ValueError, match="row_mask"):
        pkg.tree_pack(par, cu, ctx, mask[:, 0], pos)
    out = torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="row_tok"):
        pkg.accept_tree(par.long(), par, cu, par, torch.zeros(2, 5, dtype=i32), torch.zeros(2, 4, dtype=i32), out, out)
    with pytest.raises(ValueError, match="512"):
        pkg.TreeStep(1, 4, 8, 2, 600, 513)


# ------------------------------------------------------------------ on the GPU
CASES = [([1], "mixed"), ([9], "mixed"), ([64, 65, 1, 63], "mixed"), ([0, 5, 0, 17, 0], "mixed"),
         ([512, 300], "mixed"), ([512], "chain"), ([200], "star"), ([40, 130], "forest"),
         ([7] * 200, "mixed")]


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,kind", CASES)
def test_pack(pkg, sizes, kind):
    rng = np.random.default_rng(len(sizes) + sum(sizes))
    cu, parent = forest(sizes, rng, kind)
    B, live, words = len(sizes), int(cu[-1]), -(-max(max(sizes), 1) // 64)
    rows = live + 5
    ctx = rng.integers(0, 200000, B).astype(np.int32)
    full = np.concatenate([parent, np.full(5, 99, np.int32)])
    mask = torch.full((rows, words), -77, dtype=torch.int64, device="cuda")
    pos = torch.full((rows,), -77, dtype=torch.int32, device="cuda")
    pkg.tree_pack(*(torch.tensor(x, device="cuda") for x in (full, cu, ctx)), mask, pos)
    assert pkg.read_device_error() == 0
    want, wpos = O.tree_masks(parent, cu, ctx, words)
    np.testing.assert_array_equal(mask.cpu().numpy().view(np.uint64)[:live], want)
    np.testing.assert_array_equal(pos.cpu().numpy()[:live], wpos)
    assert (mask[live:] == -77).all() and (pos[live:] == -77).all()


@pytest.mark.gpu
def test_pack_bad_input(pkg):
    def run(parent, cu, ctx, words=1, rows=None):
        rows = rows or len(parent)
        t = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (parent, cu, ctx)]
        mask = torch.full((rows, words), -77, dtype=torch.int64, device="cuda")
        pos = torch.full((rows,), -77, dtype=torch.int32, device="cuda")
        pkg.tree_pack(*t, mask, pos)
        return pkg.read_device_error(), mask[:, 0].tolist(), pos.tolist()

    # a parent at or behind its row, or below -1, counts as none
    assert run([-1, 1, 0, -5], [0, 4], [10]) == (0x10, [1, 2, 5, 8], [10, 10, 11, 10])
    assert run([-1, 0], [0, 3], [10]) == (0x1, [-77] * 2, [-77] * 2)
    assert run([-1, 0, -1], [2, 0, 3], [10, 20])[0] == 0x10
    assert run([-1, 0, -1], [-1, 2, 3], [10, 20]) == (0x10, [-77, -77, 1], [-77, -77, 20])
    assert run([-1, -1], [0, 1, 2], [-1, 7]) == (0x10, [-77, 1], [-77, 7])
    assert run([-1, -1], [0, 1, 2], [2 ** 31 - 1, 7]) == (0x10, [-77, 1], [-77, 7])
    e, m, _ = run(list(range(-1, 64)), [0, 65], [0])          # 65 rows, one word
    assert e == 0x10 and m == [-77] * 65


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,kind", CASES)
@pytest.mark.parametrize("gamma", [1, 16, 32])
def test_accept(pkg, sizes, kind, gamma):
    rng = np.random.default_rng(gamma + sum(sizes))
    cu, parent = forest(sizes, rng, kind)
    live = int(cu[-1])
    tok = rng.integers(0, 4, live).astype(np.int32)            # the same token among siblings, too
    say = rng.integers(-1 if gamma == 32 else 0, 4, live).astype(np.int32)
    want = O.accept_tree(tok, parent, say, cu, gamma)
    B = len(sizes)
    out = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((B, gamma + 1), (B, gamma), (B,), (B,))]
    pkg.accept_tree(*(torch.tensor(x, device="cuda") for x in (tok, parent, cu, say)), *out)
    assert pkg.read_device_error() == 0
    for a, b in zip(out, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["chain", "mixed"])
@pytest.mark.parametrize("gamma", [4, 32])
def test_accept_walks_far(pkg, kind, gamma):
    """Every sample is the token of the row's last child: the walk ends at a leaf or at gamma."""
    cu, parent = forest([512, 300, 40, 1], np.random.default_rng(0), kind)
    tok = np.arange(int(cu[-1]), dtype=np.int32)[::-1].copy()
    say = np.full(int(cu[-1]), 9999, np.int32)
    for r in range(4):
        for i in range(int(cu[r + 1] - cu[r])):
            if parent[cu[r] + i] >= 0:
                say[cu[r] + parent[cu[r] + i]] = tok[cu[r] + i]
    want = O.accept_tree(tok, parent, say, cu, gamma)
    out = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((4, gamma + 1), (4, gamma), (4,), (4,))]
    pkg.accept_tree(*(torch.tensor(x, device="cuda") for x in (tok, parent, cu, say)), *out)
    for a, b in zip(out, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


@pytest.mark.gpu
def test_accept_bad_input(pkg):
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((2, 3), (2, 2), (2,), (2,))]
    # the second segment passes the rows there are: nothing is written
    pkg.accept_tree(t([1, 2]), t([-1, 0]), t([0, 1, 3]), t([2, 2]), *out)
    assert pkg.read_device_error() == 0x1 and all((x == -77).all() for x in out)
    # one that falls counts as empty; a parent behind its row is never taken
    pkg.accept_tree(t([1, 2, 2]), t([-1, 2, 0]), t([1, 0, 3]), t([2, 2, 5]), *out)
    assert pkg.read_device_error() == 0x10
    assert out[2].tolist() == [-1, 1] and out[0].tolist() == [[-1] * 3, [0, 2, -1]] and out[3].tolist() == [-1, 5]


def _state(rng, sizes, page, Hkv, gamma):
    B = len(sizes)
    ctx = rng.integers(0, 5 * page, B).astype(np.int32)
    ctx[0] = 2 * page                                          # the next row opens a page
    width = int(ctx.max()) // page + 3 + gamma // page
    need = -(-ctx // page)
    n_pages = int(need.sum()) + B * (2 + gamma // page) + 4
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, width), -3, np.int32)
    at = 0
    for r in range(B):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += need[r]
    return dict(page_table=table, ctx_len=ctx, anchor=np.arange(B, dtype=np.int32) + 1000,
                free_pages=perm[at:].copy(), free_top=np.array([n_pages - at], np.int32),
                k_cache=rng.integers(0, 1 << 15, (n_pages, page, Hkv, 128)).astype(np.int16),
                v_cache=rng.integers(0, 1 << 15, (n_pages, page, Hkv, 128)).astype(np.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("sizes,page,Hkv,gamma", [([9], 16, 8, 8), ([0, 30, 64, 1, 17], 16, 2, 16),
                                                  ([12] * 150, 64, 1, 32), ([200, 0], 32, 3, 4)])
def test_commit_of_a_path(pkg, sizes, page, Hkv, gamma):
    rng = np.random.default_rng(page + gamma)
    cu, parent = forest(sizes, rng)
    live, B = int(cu[-1]), len(sizes)
    tok, say = (rng.integers(0, 3, live).astype(np.int32) for _ in range(2))
    path, ptok, n, out = O.accept_tree(tok, parent, say, cu, gamma)
    assert n.max() >= 1
    s = _state(rng, sizes, page, Hkv, gamma)
    kn, vn = (rng.integers(0, 1 << 15, (live, Hkv, 128)).astype(np.int16) for _ in range(2))
    want = O.compact_path(kn, vn, cu, path, ptok, n, out, page, s["page_table"], s["ctx_len"], s["anchor"],
                          s["free_pages"], s["free_top"][0], s["k_cache"], s["v_cache"])
    d = {k: torch.tensor(v, device="cuda") for k, v in s.items()}
    g = [torch.tensor(x, device="cuda") for x in (kn, vn, cu, n, out, ptok)]
    com = torch.zeros(B, gamma + 1, dtype=torch.int32, device="cuda")
    ncom = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkg.compact_workspace_size(B), dtype=torch.uint8, device="cuda")
    pkg.compact(*g, d["page_table"], d["ctx_len"], d["anchor"], d["free_pages"], d["free_top"], d["k_cache"],
                d["v_cache"], com, ncom, ws, path=torch.tensor(path, device="cuda"))
    assert pkg.read_device_error() == 0
    for k in ("page_table", "ctx_len", "anchor", "k_cache", "v_cache"):
        np.testing.assert_array_equal(d[k].cpu().numpy(), want[k], err_msg=k)
    assert int(d["free_top"]) == want["free_top"]
    np.testing.assert_array_equal(com.cpu().numpy(), want["committed"])
    np.testing.assert_array_equal(ncom.cpu().numpy(), want["n_committed"])


@pytest.mark.gpu
@pytest.mark.parametrize("bad", ["entry", "negative", "length", "below", "rows", "ctx", "far"])
def test_commit_refused_changes_nothing(pkg, bad):
    rng = np.random.default_rng(3)
    sizes, gamma = [4, 4], 3
    cu, _ = forest(sizes, rng)
    s = _state(rng, sizes, 16, 2, gamma)
    path = np.array([[0, 2, -1, -1], [0, 1, 3, -1]], np.int32)
    n, ptok = np.array([1, 2], np.int32), np.full((2, gamma), 5, np.int32)
    if bad == "entry":
        path[1, 2] = 4
    if bad == "negative":
        path[1, 1] = -1
    if bad == "length":
        n[0] = gamma + 1
    if bad == "below":
        n[0] = -2
    if bad == "rows":
        cu = np.array([0, 9, 8], np.int32)
    if bad == "ctx":
        s["ctx_len"][1] = -100
    if bad == "far":
        s["ctx_len"][1] = 2 ** 31 - 2
    d = {k: torch.tensor(v, device="cuda") for k, v in s.items()}
    kn = torch.ones(8, 2, 128, dtype=torch.int16, device="cuda")
    out = torch.zeros(2, dtype=torch.int32, device="cuda")
    com = torch.full((2, gamma + 1), -9, dtype=torch.int32, device="cuda")
    ncom = torch.full((2,), -9, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkg.compact_workspace_size(2), dtype=torch.uint8, device="cuda")
    pkg.compact(kn, kn, torch.tensor(cu, device="cuda"), torch.tensor(n, device="cuda"), out,
                torch.tensor(ptok, device="cuda"), d["page_table"], d["ctx_len"], d["anchor"], d["free_pages"],
                d["free_top"], d["k_cache"], d["v_cache"], com, ncom, ws, path=torch.tensor(path, device="cuda"))
    assert pkg.read_device_error() == 0x10
    for k, v in s.items():
        np.testing.assert_array_equal(d[k].cpu().numpy(), v, err_msg=k)
    assert (com == -9).all() and (ncom == -9).all()


@pytest.mark.gpu
def test_accept_ends_before_a_row_without_a_sample(pkg):
    """Samples of -1: the anchor's leaves the request as it is, a later row's is not passed."""
    cu = np.array([0, 4, 8, 12, 13], np.int32)
    parent = np.array([-1, 0, 1, 1] * 3 + [-1], np.int32)
    tok = np.array([9, 5, 6, 7] * 3 + [9], np.int32)
    say = np.array([-1, 6, 1, 1, 5, -1, 1, 1, 5, 7, -1, -1, -1], np.int32)
    out = [torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((4, 4), (4, 3), (4,), (4,))]
    pkg.accept_tree(*(torch.tensor(x, device="cuda") for x in (tok, parent, cu, say)), *out)
    assert pkg.read_device_error() == 0
    path, ptok, n, last = (x.tolist() for x in out)
    assert n == [-1, 0, 1, -1] and last == [-1, 5, 7, -1]
    assert path == [[-1] * 4, [0, -1, -1, -1], [0, 1, -1, -1], [-1] * 4]
    assert ptok == [[-1] * 3, [-1] * 3, [5, -1, -1], [-1] * 3]
    for a, b in zip(out, O.accept_tree(tok, parent, say, cu, 3)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def test_alignment_refusals(pkg):
    """Addresses that a kernel's wide accesses could not take, refused before any launch."""
    lib, f, by1, by4 = pkg.load(), ctypes.c_void_p(4096), ctypes.c_void_p(4097), ctypes.c_void_p(4100)
    assert lib.dspark_tree_pack(f, f, f, 2, 8, 1, by4, f, None) == -1

    def attn(mask=f, lse=f):
        return lib.dspark_verify_attn_tree(f, f, f, f, f, 9, f, 4, f, f, mask, 1, 2, 8, 8, 2, 16,
                                           ctypes.c_float(0.1), 8, 4, f, lse, f, 1 << 40, None)

    def draw(e=f, tok=f, entry=lib.dspark_sample):
        return entry(f, 100, 0, 4, 100, f, None, 2, f, f, f, f, e, tok, f, 0, None)

    assert attn(mask=by4) == -1 and attn(lse=by1) == -1
    assert draw(e=by1) == -1 and draw(tok=by1) == -1 and draw(e=by1, entry=lib.dspark_sample_every_row) == -1
