"""Sampling from logits (dspark_sample) against its definition in fp64: kept sets and tokens exactly,
probabilities within the arithmetic's bound, and refusals.

Probabilities, for a token x octaves of w below the largest: (l_max - l) * s has three roundings, so
w is off by ln 2 * 3 * 2^-24 x relative, its exponential by 2^-21; the normaliser by the same, weighted,
and the sum of each thread's tokens (at most n) by n 2^-24; the division and the product 2^-22.  Then
one rounding to the output's type, half a step (eps / 2); fp32 numbers below 2^-126 may be 0."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O

TOP = {torch.float32: np.finfo(np.float32).max, torch.bfloat16: float(torch.finfo(torch.bfloat16).max)}


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import speculative_decoding_verification_dspark_gb300 as p
    return p


# ------------------------------------------------------------------ refusals and pins (CPU)
def test_oracle_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.1, 0.4], np.float64)).astype(np.float32)
    kept = lambda *a: list(np.flatnonzero(O.sample_row(l, *a)[1]))  # noqa: E731
    assert kept(1, 0, 1, 0) == [0, 1, 2, 3]
    assert kept(1, 3, 1, 0) == [0, 1, 3]               # the lower index of two equals
    assert kept(1, 1, 1, 0) == [1] and kept(0, 0, 1, 0) == [1]
    assert kept(1, 0, 0.79, 0) == [1, 3] and kept(1, 0, 0.85, 0) == [0, 1, 3]
    assert kept(1, 0, 0.0, 0) == [1]
    assert kept(1, 0, 1, 0.5) == [1, 3] and kept(1, 0, 1, 2.0) == [1, 3]
    assert kept(1, 3, 0.5, 0) == [1, 3]                # half of what the three hold
    t, p = O.sample_row(l, 1, 2, 1, 0, noise=np.array([1e-3, 1, 1e-3, 0.5], np.float32))
    assert t == 3 and np.allclose(p, [0, 0.5, 0, 0.5])
    assert O.sample_row(np.full(3, -np.inf, np.float32), 1, 0, 1, 0)[0] == -1


def test_host_refusals(pkg):
    lib, f, off = pkg.load(), ctypes.c_void_p(4096), ctypes.c_void_p(4097)

    def call(l=f, stride=100, dt=0, rows=4, V=100, req=f, n=None, B=2, e=f, tok=f, probs=f, pdt=0):
        return lib.dspark_sample(l, stride, dt, rows, V, req, n, B, f, f, f, f, e, tok, probs, pdt, None)

    for bad in (dict(l=None), dict(l=off), dict(probs=off), dict(stride=99), dict(dt=2), dict(pdt=2),
                dict(rows=0), dict(V=0), dict(B=0), dict(req=None), dict(e=None), dict(tok=None, probs=None),
                dict(rows=(1 << 26) + 1)):
        assert call(**bad) == -1, bad
    assert call(V=400001, stride=400001) == -2


def test_binding_refusals(pkg):
    l, e = torch.zeros(4, 100), torch.zeros(4, 100)
    tok, f2 = torch.zeros(4, dtype=torch.int32), torch.ones(2)
    with pytest.raises(ValueError, match="current CUDA device"):
        pkg.sample(l, None, None, None, None, e, tok)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        pkg.sample(l.half(), None, None, None, None, e, tok)
    with pytest.raises(ValueError, match="dense"):
        pkg.sample(l[:, ::2], None, None, None, None, e, tok)
    with pytest.raises(ValueError, match="rows, V"):
        pkg.sample(l[0], None, None, None, None, e, tok)
    del f2


# ------------------------------------------------------------------ on the GPU
def logits_of(kind, rows, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, V, generator=g)
    if kind == "wide":
        x = 3 * x
    elif kind == "narrow":
        x = 0.01 * x
    elif kind == "equal":
        x = torch.full_like(x, -1.25)
    elif kind == "two":                       # two values, many of each
        x = torch.where(x > 0.5, 2.0, -1.0)
    elif kind == "peaked":
        x = 2 * x
        x[:, V // 2] += 20
    elif kind == "masked":                    # most of the vocabulary ruled out
        x = torch.where(x > 1.2, 4 * x, torch.tensor(-float("inf")))
        x[:, V - 1] = 1.0
    elif kind == "far":                       # weights that underflow, and huge logits
        x = 1e4 * x
    elif kind == "zeros":                     # signed zeros are equal
        x = torch.where(x > 0, 0.0, -0.0)
    return x.to(dtype)


def run(pkg, logits, par, seed, probs_dtype=torch.float32, tokens=True, req=None, pad=0):
    rows, V = logits.shape
    g = torch.Generator().manual_seed(seed + 1000)
    u = torch.randint(0, 1 << 23, (rows, V), generator=g)
    noise = -torch.log((2 * u + 1).double() * 2.0 ** -24).float()
    store = torch.full((rows, V + pad), float("nan"), dtype=logits.dtype, device="cuda")
    store[:, :V] = logits.cuda()
    t, k, p, q = par
    dev = lambda x, d: None if x is None else torch.tensor(x, dtype=d, device="cuda")  # noqa: E731
    tok = torch.full((rows,), -77, dtype=torch.int32, device="cuda") if tokens else None
    pr = None if probs_dtype is None else torch.full((rows, V), 77.0, dtype=probs_dtype, device="cuda")
    f32 = torch.float32
    pkg.sample(store[:, :V], dev(t, f32), dev(k, torch.int32), dev(p, f32), dev(q, f32),
               noise.cuda() if tokens else None, tok, pr, row_req=dev(req, torch.int32))
    torch.cuda.synchronize()
    return tok, pr, noise


def compare(pkg, logits, par, seed, probs_dtype=torch.float32, pad=0):
    rows, V = logits.shape
    tok, pr, noise = run(pkg, logits, par, seed, probs_dtype, pad=pad)
    assert pkg.read_device_error() == 0
    only, _, _ = run(pkg, logits, par, seed, None, pad=pad)
    assert torch.equal(tok, only)             # the same tokens without the distributions
    tok = tok.cpu().numpy()
    f = lambda x, i, d: np.float32(d) if x is None else np.float32(x[i])  # noqa: E731
    for i in range(rows):
        l = logits[i].float().numpy()
        T, k = f(par[0], i, 1), 0 if par[1] is None else par[1][i]
        want, w = O.sample_row(l, T, k, f(par[2], i, 1), f(par[3], i, 0), noise[i].numpy(), TOP[logits.dtype])
        assert tok[i] == want, (i, tok[i], want)
        if pr is None:
            continue
        got = pr[i].double().cpu().numpy()
        with np.errstate(divide="ignore", invalid="ignore"):
            x = np.where(w > 0, np.log2(w.max() / np.where(w > 0, w, 1)), 0)
        est = np.log(2) * 3 * 2.0 ** -24
        rel = est * x + est * (w * x).sum() + 2 * 2.0 ** -21 + 2.0 ** -22 + (V // 512 + 1) * 2.0 ** -24
        tol = w * (rel + torch.finfo(probs_dtype).eps / 2) + (w > 0) * 2.0 ** -125
        bad = np.abs(got - w) > tol           # where w is 0, exactly 0
        assert not bad.any(), (i, np.flatnonzero(bad)[:5], got[bad][:5], w[bad][:5])


PARAMS = {
    "off": lambda n: (None, None, None, None),
    "heat": lambda n: ([0.1 + 0.3 * i for i in range(n)], None, None, None),
    "greedy": lambda n: ([0.0] * n, [7] * n, [0.5] * n, None),
    "top_k": lambda n: (None, [1 + 13 * i * i for i in range(n)], None, None),
    "top_p": lambda n: ([0.7] * n, None, [0.05 + 0.95 * i / n for i in range(n)], None),
    "near_one": lambda n: (None, None, [1 - 2.0 ** -(8 + 3 * i) for i in range(n)], None),
    "min_p": lambda n: (None, None, None, [1.5 * 10.0 ** -i for i in range(n)]),
    "all": lambda n: ([0.5 + 0.2 * i for i in range(n)], [3 + 400 * i for i in range(n)],
                      [0.3 + 0.15 * i for i in range(n)], [0.1 ** (i + 1) for i in range(n)]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["wide", "narrow", "equal", "two", "peaked", "masked", "far", "zeros"])
@pytest.mark.parametrize("params", list(PARAMS))
def test_kinds_and_filters(pkg, dtype, kind, params):
    n, V = 5, 5003
    compare(pkg, logits_of(kind, n, V, dtype, 1), PARAMS[params](n), 2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 511, 1024, 19456, 19457, 38912, 50257, 151936, 200001])
@pytest.mark.parametrize("params", ["off", "top_k", "top_p", "all"])
def test_vocabularies(pkg, dtype, V, params):
    compare(pkg, logits_of("wide", 4, V, dtype, V), PARAMS[params](4), V)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["equal", "narrow", "two", "wide"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_brackets(pkg, kind, dtype):
    """Ties and near ties by the ten thousand, over several CTAs."""
    n, V = 6, 100003
    x = logits_of(kind, n, V, dtype, 3)
    compare(pkg, x, (None, [1, 1024, 1025, 50000, V - 1, V], None, None), 4)
    compare(pkg, x, (None, None, [1e-6, 0.01, 0.3, 0.5, 0.9, 0.999999], None), 5)
    compare(pkg, x, (None, [40000, 60000, 3000, 2, 90000, 0], [0.5, 0.9, 0.3, 0.5, 0.99, 0.7], None), 6)


@pytest.mark.gpu
@pytest.mark.parametrize("probs_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_types_and_strides(pkg, dtype, probs_dtype, pad):
    for V in (1000, 33333):
        compare(pkg, logits_of("wide", 7, V, dtype, pad), PARAMS["all"](7), 8, probs_dtype, pad)


@pytest.mark.gpu
def test_borders_that_fp32_cannot_tell(pkg):
    """Equal weights: the mass before token i is i / V exactly, and top-p meets it to 2^-24."""
    V = 4096
    x = torch.zeros(6, V)
    at = [1024 / V, 1024 / V + 2.0 ** -26, 1024 / V - 2.0 ** -26, 0.5, 0.5 - 2.0 ** -25, 0.5 + 2.0 ** -24]
    compare(pkg, x, (None, None, at, None), 9)
    x[:, ::2] = -0.5
    compare(pkg, x, (None, None, at, None), 9)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [700, 1000, 5000])
def test_borders_of_top_p_within_top_k(pkg, V):
    """Top-p meets a border exactly among the tokens that top-k leaves, the list holding them all."""
    n = 6
    x = torch.full((n, V), -30.0)
    x[:, 1:V:V // 640] = 0.5                    # some 640 and more equal ones
    k = [64, 100, 128, 500, 600, 640]
    for p in (0.5, 0.25, 0.75):
        compare(pkg, x, (None, k, [p] * n, None), 12)
        compare(pkg, x.bfloat16(), (None, k, [p] * n, None), 12)


@pytest.mark.gpu
def test_special_values(pkg):
    for dtype in (torch.float32, torch.bfloat16):
        x = logits_of("wide", 6, 3001, dtype, 1)
        x[0, 5] = float("nan")
        x[1, [7, 9]] = float("inf")
        x[2] = -float("inf")
        x[2, 1234] = -5
        x[3] = float("nan")
        x[3, 4] = float("inf")
        x[4, :1500] = -float("inf")
        x[5] = -torch.finfo(dtype).max
        for params in ("off", "top_k", "top_p", "all"):
            compare(pkg, x, PARAMS[params](6), 3)


@pytest.mark.gpu
def test_rows_without_a_token(pkg):
    x = torch.full((3, 70001), -float("inf"))
    x[1] = float("nan")
    x[2, 69999] = 0.0
    tok, pr, _ = run(pkg, x, (None, [2, 2, 2], [0.5] * 3, None), 1)
    assert pkg.read_device_error() == 0
    assert tok.tolist() == [-1, -1, 69999]
    assert (pr[:2] == 0).all() and pr[2, 69999] == 1 and pr[2].sum() == 1


@pytest.mark.gpu
def test_ties_of_the_race_go_to_the_lowest_index(pkg):
    x = torch.zeros(2, 60000, device="cuda")
    e = torch.full((2, 60000), 0.5, device="cuda")
    e[1, [31000, 59000]] = 0.25
    tok = torch.zeros(2, dtype=torch.int32, device="cuda")
    pkg.sample(x, None, None, None, None, e, tok)
    assert tok.tolist() == [0, 31000]


@pytest.mark.gpu
def test_padding_rows_and_shared_parameters(pkg):
    x = logits_of("wide", 6, 2000, torch.float32, 5)
    req = [0, 0, -1, 1, 1, -1]
    par = ([0.5, 1.5], [10, 0], [1.0, 0.8], [0.0, 0.0])
    tok, pr, noise = run(pkg, x, par, 7, req=req)
    assert pkg.read_device_error() == 0
    for i, r in enumerate(req):
        if r < 0:
            assert tok[i] == -77 and (pr[i] == 77).all()
            continue
        f = [np.float32(p[r]) for p in par]
        want, w = O.sample_row(x[i].numpy(), f[0], par[1][r], f[2], f[3], noise[i].numpy())
        assert int(tok[i]) == want
        np.testing.assert_array_equal(pr[i].cpu().numpy() > 0, w > 0)


@pytest.mark.gpu
def test_bad_parameters_leave_the_row(pkg):
    x = logits_of("wide", 5, 300, torch.float32, 5)
    bad = [0.5, -1.0, float("nan"), float("inf"), 2.0 ** -70]
    tok, pr, _ = run(pkg, x, (bad, None, None, None), 1)
    assert pkg.read_device_error() == 0x10
    assert tok[0] >= 0 and tok[1:].tolist() == [-77] * 4 and (pr[1:] == 77).all()
    tok, pr, _ = run(pkg, x, ([1.0], None, None, None), 1, req=[0, 1, 0, 0, 0])
    assert pkg.read_device_error() == 0x10 and tok[1] == -77 and tok[0] >= 0
    tok, pr, _ = run(pkg, x, (None, None, [0.5, float("nan"), 0.5, 0.5, 0.5], None), 1)
    assert pkg.read_device_error() == 0x10 and tok[1] == -77 and tok[0] >= 0


@pytest.mark.gpu
def test_draws_follow_the_distribution(pkg):
    V, n = 5, 20000
    x = torch.log(torch.tensor([0.1, 0.2, 0.3, 0.15, 0.25])).repeat(n, 1)
    tok, _, _ = run(pkg, x, (None, None, None, None), 11, None)
    got = torch.bincount(tok.cpu().long(), minlength=V) / n
    # five standard deviations of a frequency
    assert (got - torch.tensor([0.1, 0.2, 0.3, 0.15, 0.25])).abs().max() < 5 * (0.25 / n) ** 0.5


@pytest.mark.gpu
def test_rows_from_n_rows_on_are_left(pkg):
    x = logits_of("wide", 6, 40000, torch.float32, 5).cuda()
    e = torch.full((6, 40000), 0.5, device="cuda")
    full = torch.zeros(6, dtype=torch.int32, device="cuda")
    pkg.sample(x, None, None, None, None, e, full)
    for n in (0, 3, 6, 99):
        tok = torch.full((6,), -77, dtype=torch.int32, device="cuda")
        pkg.sample(x, None, None, None, None, e, tok, n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert torch.equal(tok[:n], full[:n]) and (tok[n:] == -77).all()
    assert pkg.read_device_error() == 0


@pytest.mark.gpu
def test_calls_on_two_streams(pkg):
    """Two calls at once, and a call on a stream whose inputs another one wrote."""
    x = [logits_of("wide", 40, 70001, torch.bfloat16, i).cuda() for i in range(2)]
    e = torch.rand(40, 70001, device="cuda") + 0.01
    p = torch.full((40,), 0.9, device="cuda")
    want = []
    for y in x:
        want.append(torch.zeros(40, dtype=torch.int32, device="cuda"))
        pkg.sample(y, None, None, p, None, e, want[-1])
    torch.cuda.synchronize()
    got = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in x]
    for _ in range(3):
        for s, y, t in zip(streams, x, got):
            with torch.cuda.stream(s):
                pkg.sample(y, None, None, p, None, e, t)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def _over_ctas(kind, n, V, dtype, seed):
    """n rows and a temperature: logits that lie so close that no list holds those around the k-th, or
    more equal largest ones than a list holds, in one part of the row alone."""
    g = torch.Generator().manual_seed(seed)
    x, T = torch.randn(n, V, generator=g), 1.0
    at, size = {"first": (0, V // 8), "middle": (3 * V // 8 + 5, V // 8), "last": (V - V // 8, V // 8),
                "most": (0, V // 4 + 3)}.get(kind, (0, 0))
    if kind == "narrow":
        x = 0.001 * x
    elif kind in ("hot", "hotter"):
        x, T = 3 * x, 1e3 if kind == "hot" else 1e6
    elif kind == "masked":                    # all ruled out but one range, of nearly equal ones
        x = 0.001 * x
        x[:, :V // 2], x[:, V // 2 + 4000:] = -float("inf"), -float("inf")
    else:
        x = x.clamp(max=4.0) - (10.0 if kind == "most" else 0.0)
        x[:, at:at + size] = 5.0
    return x.to(dtype), T


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["first", "middle", "last", "most", "masked", "narrow", "hot", "hotter"])
@pytest.mark.parametrize("V,dtype", [(151936, torch.float32), (129280, torch.bfloat16),
                                     (50257, torch.float32), (50257, torch.bfloat16)])
def test_short_top_k_over_several_ctas(pkg, kind, V, dtype):
    """Where the k-th lies among thousands, all CTAs of a row search the same range for it."""
    k = [1, 2, 50, 73, 100, 133, 200, 231, 400, 512]
    n = len(k)
    x, T = _over_ctas(kind, n, V, dtype, V)
    compare(pkg, x, ([T] * n, k, None, None), 13)
    compare(pkg, x, ([T] * n, k, [0.05 + 0.09 * i for i in range(n)], [0.3, 0.9] * (n // 2)), 14, None)


@pytest.mark.gpu
def test_top_p_of_zero_over_several_ctas(pkg):
    """The first token alone, among thousands of equal ones."""
    x, _ = _over_ctas("most", 4, 151936, torch.float32, 1)
    compare(pkg, x, (None, None, [0.0, -1.0, 0.0, 0.5], None), 15)


def _race(pkg, logits, noise, T, kind):
    """Tokens of the call with and without distributions, and what the oracle draws."""
    rows, V = logits.shape
    dev = lambda x: None if x is None else torch.full((rows,), x, device="cuda")  # noqa: E731
    got = []
    for probs in (None, torch.zeros(rows, V, device="cuda")):
        tok = torch.full((rows,), -77, dtype=torch.int32, device="cuda")
        pkg.sample(logits.cuda(), dev(T), None, dev(0.999 if kind == "top_p" else None), None, noise.cuda(), tok, probs)
        got.append(tok.tolist())
    assert pkg.read_device_error() == 0
    p = np.float32(0.999 if kind == "top_p" else 1)
    return got, [O.sample_row(l.float().numpy(), np.float32(T), 0, p, np.float32(0), e.numpy())[0]
                 for l, e in zip(logits, noise)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["off", "top_p"])
@pytest.mark.parametrize("V", [3000, 60000, 151936])
def test_near_ties_of_the_race(pkg, V, kind):
    """Many tokens whose scores are one fp32 number, or apart by less than its error: the winner is
    the definition's, wherever it stands among them."""
    g = torch.Generator().manual_seed(V)
    # different logits of one fp32 weight, constant noise
    x = 1 + torch.randint(0, 64, (4, V), generator=g) * 2.0 ** -20
    for i in range(4):
        x[i, (2 * i + 1) * V // 8] = 1 + 64 * 2.0 ** -20
    got, want = _race(pkg, x, torch.full((4, V), 0.5), 1e5, kind)
    assert got == [want] * 2
    # 20 to 90 octaves below the largest, with noise that brings them to a score of 1 +- 2^-24
    x = -14 - 48 * torch.rand(4, V, generator=g)
    x[:, 5] = 0.0
    noise = torch.exp(x.double()).float()
    noise[:, 5] = 4.0
    got, want = _race(pkg, x, noise, 1.0, "off")
    assert got == [want] * 2


@pytest.mark.gpu
@pytest.mark.parametrize("V,dtype", [(151936, torch.float32), (38000, torch.bfloat16)])
def test_borders_of_top_p_with_a_common_error(pkg, V, dtype):
    """Half the mass in equal logits far below the top, whose weights share one rounding error: the whole
    is off by some 2^-21 in fp32.  Top-p meets the mass before a token between them to 2^-25."""
    rng, n = np.random.default_rng(V), 32
    x, T, p = torch.zeros(n, V), [], []
    f32, bf = np.float32, lambda a: torch.tensor(a, dtype=torch.float32).to(dtype).float().numpy()  # noqa: E731
    for r in range(n):
        octaves = np.log2(V)
        t = rng.uniform(0.6, 1.9, 400).astype(f32)
        # of many temperatures and values those whose exponent is rounded farthest, up or down
        c = (f32(1.442695) / t)[:, None]
        l = bf(-np.log(2) * octaves * t[:, None] * rng.uniform(0.99, 1.01, (400, 400)))
        err = (-l * c).astype(np.float64) + l.astype(np.float64) / np.log(2) / t[:, None]
        at = np.unravel_index((err if r % 2 else -err).argmax(), err.shape)
        T.append(float(t[at[0]]))
        row = np.full(V, l[at], f32)
        some = rng.permutation(V)[:301]
        row[some[0]] = 0
        mid = bf(-np.log(2) * (octaves - 1) * T[-1] * np.linspace(0.98, 1.02, 300))
        row[some[1:]] = mid
        x[r] = torch.tensor(row)
        e = np.exp(np.sort(row.astype(np.float64))[::-1] / T[-1])
        before, i = e.cumsum() - e, 100 + 3 * r
        q = f32(before[i] / e.sum())
        while r % 4 < 2 and float(q) * e.sum() >= before[i]:
            q = np.nextafter(q, f32(0))
        while r % 4 >= 2 and float(q) * e.sum() <= before[i]:
            q = np.nextafter(q, f32(1))
        p.append(float(q))
    compare(pkg, x.to(dtype), (T, None, p, None), 16)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [300, 70001])
def test_every_row_is_written(pkg, V):
    """Refused and padding rows before n_rows get token -1 and no probability."""
    x = logits_of("wide", 6, V, torch.float32, 5).cuda()
    dev = lambda v, d: torch.tensor(v, dtype=d, device="cuda")  # noqa: E731
    e = torch.full((6, V), 0.5, device="cuda")
    T, req = dev([1.0, float("nan"), -1.0], torch.float32), dev([0, 1, -1, 2, 7, 0], torch.int32)
    out = []
    for every in (False, True):
        tok = torch.full((6,), -77, dtype=torch.int32, device="cuda")
        pr = torch.full((6, V), 77.0, device="cuda")
        pkg.sample(x, T, None, None, None, e, tok, pr, req, n_rows=dev([5], torch.int32), every_row=every)
        assert pkg.read_device_error() == 0x10
        out.append((tok, pr))
    first = int(out[0][0][0])
    assert first >= 0 and out[0][0].tolist() == [first] + [-77] * 5 and (out[0][1][1:] == 77).all()
    assert out[1][0].tolist() == [first] + [-1] * 4 + [-77]
    assert torch.equal(out[0][1][0], out[1][1][0]) and (out[1][1][1:5] == 0).all() and (out[1][1][5] == 77).all()


@pytest.mark.gpu
def test_request_indices_without_parameters(pkg):
    """A few rows of a large batch: no parameter is read, so an index past the rows is none out of range."""
    x = logits_of("wide", 3, 500, torch.float32, 5).cuda()
    e = torch.full((3, 500), 0.5, device="cuda")
    want, tok = (torch.full((3,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    pkg.sample(x, None, None, None, None, e, want)
    pkg.sample(x, None, None, None, None, e, tok, row_req=torch.tensor([9, -1, 1000], dtype=torch.int32, device="cuda"))
    assert pkg.read_device_error() == 0
    assert tok.tolist() == [int(want[0]), -77, int(want[2])]


@pytest.mark.gpu
@pytest.mark.parametrize("V", [700, 60000])
def test_the_smallest_and_largest_top_p(pkg, V):
    p = [1e-45, 1e-38, 1e-30, 1e-12, 1 - 2.0 ** -24, 1 - 2.0 ** -23]
    for kind in ("wide", "equal", "two", "narrow"):
        compare(pkg, logits_of(kind, 6, V, torch.float32, 4), (None, None, p, None), 17)
