"""Query/key norm with the position rotation (dspark_qk_norm_rope) against the oracle's
fp64 formulas, and its refusals.

Tolerance, from the arithmetic: the output's one rounding to bf16 is at most 2^-8 of the
value.  Before it, in fp32: the sum of 128 squares (8 in a row, then 4 pairwise) errs by
less than 12 * 2^-24, its square root, the quotient and the two products by less than
6 * 2^-24, so a normed element by less than 2^-19 relative.  The angle's turns are exact
to 2^-31 * 2^-52 relative in fp64 and rounded to fp32 below half a turn (2^-26 of a turn,
2^-23 rad), sine and cosine err by 2^-22, the two products and the sum by 2^-22: an
element of the rotated pair by less than 2^-18 (|y_a| + |y_b|)."""
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
def test_oracle_position_zero_is_the_norm_alone():
    x = np.random.default_rng(0).normal(size=(1, 2, 128))
    y, _ = O.qk_norm_rope(x, np.ones(128), 0.0, [1.0] * 64, False, 1.0, [0])
    np.testing.assert_allclose(np.mean(y * y, -1), 1.0, rtol=1e-12)
    np.testing.assert_allclose(y / x, np.broadcast_to((y / x)[..., :1], y.shape), rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_scores_depend_on_the_distance_alone(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(1, 1, 128)), rng.normal(size=(1, 1, 128))
    inv = 10000.0 ** (-np.arange(64) / 64)
    dots = []
    for p in (0, 5, 1000):
        a, _ = O.qk_norm_rope(q, None, 0.0, inv, interleaved, 1.0, [p + 17])
        b, _ = O.qk_norm_rope(k, None, 0.0, inv, interleaved, 1.0, [p])
        dots.append(float(np.sum(a * b)))
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
    # a quarter turn of the first pair
    y, _ = O.qk_norm_rope(q, None, 0.0, [np.pi / 2], interleaved, 1.0, [1])
    np.testing.assert_allclose(y[0, 0, :2], [-q[0, 0, 1], q[0, 0, 0]], atol=1e-12)


# ------------------------------------------------------------------ refusals (CPU)
def test_host_refusals(pkg):
    import ctypes
    lib, f = pkg.load(), ctypes.c_void_p(4096)
    off = ctypes.c_void_p(4104)

    def call(q_in=f, qs=1024, v_in=f, v=f, dt=1, wq=f, eps=1e-6, inv=f, rot=128, rows=4, hq=8,
             hkv=2, q=f, pos=f):
        return lib.dspark_qk_norm_rope(q_in, qs, f, 256, v_in, 256, dt, wq, f, eps, inv, rot, 0,
                                       1.0, pos, None, rows, hq, hkv, q, f, v, None)

    assert call(q_in=None) == -1 and call(pos=None) == -1 and call(q=None) == -1
    assert call(v_in=None) == -1 and call(v=None) == -1          # v_in and v_new go together
    assert call(dt=2) == -1 and call(rows=0) == -1 and call(hkv=0) == -1 and call(eps=-1.0) == -1
    assert call(rot=24) == -2 and call(rot=144) == -2 and call(rot=-16) == -2
    assert call(inv=None) == -1                                  # a rotation needs frequencies
    assert call(qs=1016) == -1 and call(qs=1028) == -1           # overlapping; not 16 bytes
    assert call(q_in=off) == -1 and call(q=off) == -1 and call(wq=off) == -1


def test_binding_refusals(pkg):
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    pos = torch.zeros(4, dtype=torch.int32)
    good = [t(4, 8, 128), t(4, 2, 128), t(4, 2, 128), None, None, None, pos, t(4, 8, 128),
            t(4, 2, 128), t(4, 2, 128)]
    with pytest.raises(ValueError):      # host tensors
        pkg.qk_norm_rope(*good)
    for at, bad in ((0, t(4, 8, 128, dt=torch.float16)), (1, t(3, 2, 128)), (1, t(4, 2, 128, dt=torch.float32)),
                    (0, t(4, 128, 8).transpose(1, 2)), (2, None), (9, None)):
        a = list(good)
        a[at] = bad
        with pytest.raises(ValueError):
            pkg.qk_norm_rope(*a)


# ------------------------------------------------------------------ parity (GPU)
CASES = [  # rows, tail, hq, hkv, rotary, interleaved, dtype, fused, weights, max_pos, factor
    (1, 0, 32, 8, 128, False, "bf16", True, True, 4096, 1.0),
    (5, 3, 8, 2, 128, True, "bf16", False, True, 100, 1.0),
    (17, 0, 7, 1, 64, False, "f32", True, True, 1 << 20, 1.25),
    (33, 31, 40, 8, 32, True, "f32", False, False, 1 << 20, 1.0),
    (3, 1, 1, 1, 96, False, "bf16", False, True, 2 ** 31 - 1, 1.0),
    (9, 0, 16, 16, 16, True, "bf16", True, False, 50, 0.5),
    (4, 0, 70, 3, 0, False, "bf16", True, True, 50, 1.0),
    # groups of 2, 4, 8 and 16 rows, the last ones cut short
    (1501, 6, 9, 2, 128, False, "bf16", True, True, 9000, 1.0),
    (2503, 0, 5, 8, 64, True, "bf16", False, True, 131072, 1.0),
    (2901, 13, 3, 1, 32, True, "f32", True, True, 1 << 20, 1.0),
    (9999, 1, 1, 1, 128, False, "bf16", False, True, 2 ** 31 - 1, 1.0),
]


def _inputs(rows, tail, hq, hkv, rotary, dtype, fused, weights, max_pos, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    n = rows + tail
    parts = [(3 * torch.randn(n, h, 128, generator=g)).to(dt) for h in (hq, hkv, hkv)]
    parts[0][0, 0] = 0                       # a zero head: eps alone under the root
    pos = torch.randint(0, max_pos, (n,), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0] = max_pos - 1
    pos[rows:] = -1
    if rows > 2:
        pos[1] = -1                          # padding in the middle
    if rows > 100:
        pos[rows // 2:rows // 2 + 37] = -1
    w = [1 + 0.3 * torch.randn(128, generator=g) if weights else None for _ in range(2)]
    inv = (10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / max(rotary, 1))).float()
    dev = [p.cuda() for p in parts]
    if fused:
        f = torch.cat([p.flatten(1) for p in dev], 1)
        dev = [p.unflatten(1, (-1, 128)) for p in f.split([hq * 128, hkv * 128, hkv * 128], 1)]
    return parts, dev, pos, w, inv


def _outputs(n, hq, hkv, fill=7.0):
    return [torch.full((n, h, 128), fill, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]


def _check(parts, outs, pos, w, inv, inter, factor, eps, fill=7.0):
    live = pos.numpy() >= 0
    for x, y, wt in zip(parts[:2], outs, w):
        ref, mag = O.qk_norm_rope(x.double().numpy(), None if wt is None else wt.numpy(), eps,
                                  inv.numpy(), inter, factor, pos.numpy())
        y = y.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * mag + 1e-38
        assert np.all(np.abs(y - ref)[live] <= tol[live])
        assert np.all(y[~live] == fill)
    v = outs[2].cpu()
    assert torch.equal(v[live], parts[2].to(torch.bfloat16)[live])
    assert bool((v[~live] == fill).all())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,tail,hq,hkv,rotary,inter,dtype,fused,weights,max_pos,factor", CASES)
def test_parity(pkg, rows, tail, hq, hkv, rotary, inter, dtype, fused, weights, max_pos, factor):
    parts, dev, pos, w, inv = _inputs(rows, tail, hq, hkv, rotary, dtype, fused, weights, max_pos)
    outs = _outputs(rows + tail, hq, hkv)
    wd = [None if t is None else t.cuda() for t in w]
    pkg.qk_norm_rope(*dev, *wd, inv.cuda() if rotary else None, pos.cuda(), *outs, eps=1e-6,
                     interleaved=inter, attn_factor=factor)
    torch.cuda.synchronize()
    _check(parts, outs, pos, w, inv, inter, factor, 1e-6)


@pytest.mark.gpu
def test_rows_from_n_rows_on_and_no_values(pkg):
    parts, dev, pos, w, inv = _inputs(12, 0, 8, 2, 128, "bf16", True, True, 500)
    outs = _outputs(12, 8, 2)
    n = torch.tensor([7], dtype=torch.int32, device="cuda")
    pkg.qk_norm_rope(dev[0], dev[1], None, w[0].cuda(), w[1].cuda(), inv.cuda(), pos.cuda(),
                     outs[0], outs[1], None, n_rows=n)
    torch.cuda.synchronize()
    pos[7:] = -1
    outs[2] = torch.where((pos >= 0)[:, None, None], parts[2], torch.tensor(7.0).bfloat16()).cuda()
    _check(parts, outs, pos, w, inv, False, 1.0, 1e-6)


@pytest.mark.gpu
def test_one_weight_and_many_rows_cut_by_n_rows(pkg):
    parts, dev, pos, w, inv = _inputs(2000, 0, 4, 2, 64, "bf16", True, True, 5000)
    n = torch.tensor([1503], dtype=torch.int32, device="cuda")
    pos[1503:] = 77                          # (whatever row_pos holds there)
    for use in ((True, False), (False, True)):
        wu = [t if u else None for t, u in zip(w, use)]
        outs = _outputs(2000, 4, 2)
        pkg.qk_norm_rope(*dev, *[None if t is None else t.cuda() for t in wu], inv.cuda(), pos.cuda(),
                         *outs, interleaved=True, n_rows=n)
        torch.cuda.synchronize()
        cut = pos.clone()
        cut[1503:] = -1
        _check(parts, outs, cut, wu, inv, True, 1.0, 1e-6)


@pytest.mark.gpu
def test_in_place_other_stream_and_graph(pkg):
    parts, dev, pos, w, inv = _inputs(9, 0, 32, 8, 128, "bf16", False, True, 9000)
    wd, invd, posd = [t.cuda() for t in w], inv.cuda(), pos.cuda()
    outs = [p.clone() for p in dev]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkg.qk_norm_rope(*outs, *wd, invd, posd, *outs)
    s.synchronize()
    keep = [torch.where((posd >= 0)[:, None, None], o, torch.full_like(o, 7.0)) for o in outs]
    _check(parts, keep, pos, w, inv, False, 1.0, 1e-6)
    again = _outputs(9, 32, 8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.qk_norm_rope(*dev, *wd, invd, posd, *again)
    for _ in range(2):
        for a in again:
            a.fill_(7.0)
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, keep))


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_head(pkg):
    parts, dev, pos, w, inv = _inputs(6, 0, 8, 2, 128, "f32", False, True, 500)
    for src in (parts, dev):
        src[0][3, 2, 5] = float("nan")
        src[1][4, 1, 9] = float("inf")
    outs = _outputs(6, 8, 2)
    pkg.qk_norm_rope(*dev, w[0].cuda(), w[1].cuda(), inv.cuda(), pos.cuda(), *outs)
    torch.cuda.synchronize()
    assert bool(outs[0][3, 2].isnan().all()) and bool(outs[1][4, 1].isnan().any())
    for t, r, h in ((0, 3, 2), (1, 4, 1)):  # their heads aside, as before
        parts[t][r, h] = 1.0
        ref, _ = O.qk_norm_rope(parts[t][r:r + 1, h:h + 1].double().numpy(), w[t].numpy(), 1e-6,
                                inv.numpy(), False, 1.0, pos[r:r + 1].numpy())
        outs[t][r, h] = torch.tensor(ref[0, 0]).bfloat16().cuda()
    _check(parts, outs, pos, w, inv, False, 1.0, 1e-6)
