"""A step on trees of drafted tokens, as a program runs it (TreeStep): tree_pack, norm and rotation,
attention, sampling, the walk and the commit, against the oracle at every stage; the same captured
into a graph and on a stream of its own; and the chain's step with its distributions from logits."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import dspark_oracle as O
from tests.test_tree import _state, forest
from tests.test_verify_attn_tree import check

HQ, HKV, V, PAGE, GAMMA = 8, 2, 3001, 16, 8


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import speculative_decoding_verification_dspark_gb300 as p
    return p


def make(sizes, seed=0, pad=4):
    rng = np.random.default_rng(seed)
    cu, parent = forest(sizes, rng)
    live, B = int(cu[-1]), len(sizes)
    rows = live + pad
    s = _state(rng, sizes, PAGE, HKV, GAMMA)
    g = torch.Generator().manual_seed(seed)
    bf = lambda *x: torch.randn(*x, generator=g).bfloat16()  # noqa: E731
    d = {k: torch.tensor(v, device="cuda") for k, v in s.items() if k not in ("k_cache", "v_cache")}
    for k in ("k_cache", "v_cache"):
        d[k] = bf(*s[k].shape).cuda()
    qkv = bf(rows, (HQ + 2 * HKV) * 128).cuda()
    d["q_in"], d["k_in"], d["v_in"] = (x.unflatten(1, (-1, 128)) for x in
                                       qkv.split([HQ * 128, HKV * 128, HKV * 128], 1))
    d["q"], d["k_new"], d["v_new"] = (torch.zeros(rows, h, 128, dtype=torch.bfloat16, device="cuda")
                                      for h in (HQ, HKV, HKV))
    # tokens of few kinds, and logits that favour them: walks of some length
    tok = rng.integers(0, 3, rows).astype(np.int32)
    logits = 2 * torch.randn(rows, V, generator=g)
    logits[:, :3] += 9
    u = torch.randint(0, 1 << 23, (rows, V), generator=g)
    d.update(cu_seqlens=torch.tensor(cu, device="cuda"), row_tok=torch.tensor(tok, device="cuda"),
             row_parent=torch.tensor(np.concatenate([parent, np.full(pad, 7)]).astype(np.int32), device="cuda"),
             row_req=torch.tensor(np.concatenate([np.repeat(np.arange(B), sizes), np.zeros(pad)]).astype(np.int32),
                                  device="cuda"),
             inv_freq=(1e4 ** (-torch.arange(0, 128, 2) / 128)).float().cuda(), scale=128 ** -0.5,
             logits=logits.cuda(), exp_noise=(-torch.log((2 * u + 1).double() * 2.0 ** -24)).float().cuda(),
             temperature=torch.tensor([0.0, 0.8, 1.3][:B] * (B // 3 + 1), device="cuda")[:B].contiguous(),
             top_k=torch.tensor(([0, 20] * B)[:B], dtype=torch.int32, device="cuda"),
             top_p=torch.tensor(([1.0, 0.9, 0.95] * B)[:B], device="cuda"))
    return d, rows


STATE = ("page_table", "ctx_len", "anchor", "free_top", "k_cache", "v_cache")
OUT = ("row_mask", "row_pos", "out", "lse", "row_sample", "path", "path_tok", "accept_len", "out_tok",
       "committed", "n_committed")


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[9], [17, 0, 40], [64, 1, 33, 5, 100]])
def test_step_against_the_oracle(pkg, sizes):
    d, rows = make(sizes, seed=len(sizes))
    B, live = len(sizes), sum(sizes)
    step = pkg.TreeStep(B, GAMMA, HQ, HKV, rows, max(sizes))
    before = {k: d[k].clone() for k in STATE}
    step.run(d)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    n = lambda t: (t.float() if t.dtype == torch.bfloat16 else t).cpu().numpy()  # noqa: E731
    cu, parent = n(d["cu_seqlens"]), n(d["row_parent"])[:live]
    ctx = n(before["ctx_len"])
    mask, pos = O.tree_masks(parent, cu, ctx, step.row_mask.shape[1])
    np.testing.assert_array_equal(n(step.row_mask).view(np.uint64)[:live], mask)
    np.testing.assert_array_equal(n(step.row_pos)[:live], pos)
    want, mag = O.qk_norm_rope(d["k_in"].double().cpu().numpy()[:live], None, 1e-6, n(d["inv_freq"]), False, 1.0, pos)
    assert np.all(np.abs(n(d["k_new"])[:live] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * mag)
    check(n(step.out)[:live], n(step.lse)[:live],
          O.verify_attention_tree(n(d["q"])[:live], n(d["k_new"])[:live], n(d["v_new"])[:live],
                                  n(before["k_cache"]), n(before["v_cache"]), n(before["page_table"]), ctx, cu,
                                  mask, d["scale"]), int(ctx.max()) + max(sizes))
    req, logits, e = n(d["row_req"]), n(d["logits"]), n(d["exp_noise"])
    T, k, p = (n(d[x]) for x in ("temperature", "top_k", "top_p"))
    say = np.array([O.sample_row(logits[i], T[req[i]], k[req[i]], p[req[i]], np.float32(0), e[i])[0]
                    for i in range(live)], np.int32)
    np.testing.assert_array_equal(n(step.row_sample)[:live], say)
    walk = O.accept_tree(n(d["row_tok"])[:live], parent, say, cu, GAMMA)
    for name, w in zip(("path", "path_tok", "accept_len", "out_tok"), walk):
        np.testing.assert_array_equal(n(getattr(step, name)), w, err_msg=name)
    after = O.compact_path(n(d["k_new"]), n(d["v_new"]), cu, *walk, PAGE, n(before["page_table"]), ctx,
                           n(before["anchor"]), n(d["free_pages"]), int(before["free_top"]), n(before["k_cache"]),
                           n(before["v_cache"]))
    for x in STATE:
        np.testing.assert_array_equal(n(d[x]).reshape(-1), np.asarray(after[x]).reshape(-1), err_msg=x)
    np.testing.assert_array_equal(n(step.committed), after["committed"])
    # rows past the last are left as they are
    assert (step.out[live:] == 0).all() and (step.row_sample[live:] == 0).all() and (step.row_pos[live:] == 0).all()


@pytest.mark.gpu
def test_two_graphs_and_a_stream(pkg):
    """The step called, on a stream of its own, and replayed from two graphs that share the workspaces:
    the same bits."""
    sizes = [30, 64, 3]
    d, rows = make(sizes, seed=8)
    step = pkg.TreeStep(len(sizes), GAMMA, HQ, HKV, rows, 64)
    before = {k: d[k].clone() for k in STATE}

    def reset():
        for k in STATE:
            d[k].copy_(before[k])
        for k in OUT:
            getattr(step, k).zero_()
        torch.cuda.synchronize()

    def result():
        torch.cuda.synchronize()
        assert pkg.read_device_error() == 0
        return [getattr(step, k).clone() for k in OUT] + [d[k].clone() for k in STATE]

    reset()
    step.run(d)
    want = result()
    reset()
    side = torch.cuda.Stream()
    step.run(d, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(result(), want))
    graphs = []
    for _ in range(2):
        reset()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step.run(d)
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        reset()
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(result(), want))
    reset()
    graphs[0].replay()          # two steps, one behind the other, as called
    graphs[1].replay()
    two = result()
    reset()
    step.run(d)
    step.run(d)
    assert all(torch.equal(a, b) for a, b in zip(result(), two))


def test_graph_refuses_logits(pkg):
    step = pkg.VerifyStep(2, 4, 8, 2, 128, 128, 1024, 16, device="cpu")
    with pytest.raises(ValueError, match="logits"):
        step.graph(dict(logits=torch.zeros(16, 1024)), O.COMPACT)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [O.COMPACT, O.STATIC])
def test_chain_step_from_logits(pkg, mode):
    """VerifyStep with logits: p_target is sample's, and the step that reads it by hand gives the same."""
    import harness
    wl = W.WORKLOADS["tiny"]
    d, step = harness.prepare(W.make_inputs(wl, seed=4), mode)
    snap = harness.snapshot_state(d)
    rows = step.max_rows
    for k in ("q", "k_new", "v_new"):
        full = torch.zeros(rows, *d[k].shape[1:], dtype=d[k].dtype, device="cuda")
        full[:d[k].shape[0]] = d[k]
        d[k] = full
    g = torch.Generator().manual_seed(2)
    logits = 2 * torch.randn(rows, wl.vocab, generator=g)
    par = dict(temperature=torch.full((wl.B,), 0.7), top_p=torch.full((wl.B,), 0.9),
               top_k=torch.full((wl.B,), 100, dtype=torch.int32))
    d["p_target"] = torch.zeros(rows, wl.vocab, device="cuda")
    e = dict(d, logits=logits.cuda(), **{k: v.cuda() for k, v in par.items()})
    step.run(e, mode)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    M = int(step.M_pack)
    for i in range(M):
        w = O.sample_row(logits[i].numpy(), np.float32(0.7), 100, np.float32(0.9), np.float32(0))[1]
        got = d["p_target"][i].cpu().numpy()
        np.testing.assert_array_equal(got > 0, w > 0)
        np.testing.assert_allclose(got, w, rtol=2.0 ** -16)
    assert (d["p_target"][M:] == 0).all()
    names = ("accept_len", "out_tok", "committed", "n_committed")
    got = [getattr(step, n).clone() for n in names] + [d[k].clone() for k in ("k_cache", "ctx_len")]
    harness.restore_state(d, snap)
    step.run(d, mode)           # from that p_target
    torch.cuda.synchronize()
    want = [getattr(step, n) for n in names] + [d[k] for k in ("k_cache", "ctx_len")]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_rows_without_a_token_commit_nothing(pkg):
    """Logits that are all -inf leave a row without a sample: at an anchor the request keeps its state,
    on a path the commit ends before that row."""
    sizes = [30, 30, 30]
    d, rows = make(sizes, seed=3)
    # a chain of token 0 in the requests; every sample is token 0
    d["row_parent"][:90] = torch.tensor([-1] + list(range(29)), dtype=torch.int32, device="cuda").repeat(3)
    d["row_tok"].zero_()
    d["logits"][:] = -1.0
    d["logits"][:, 0] = 50.0
    d["logits"][30] = -float("inf")               # the second request's anchor
    d["logits"][60 + 3] = float("nan")            # the fourth row of the third's path
    step = pkg.TreeStep(3, GAMMA, HQ, HKV, rows, 30)
    ctx, anchor = d["ctx_len"].clone(), d["anchor"].clone()
    step.run(d)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    assert step.row_sample[[30, 63]].tolist() == [-1, -1]
    assert step.accept_len.tolist() == [GAMMA, -1, 2] and step.out_tok.tolist() == [0, -1, 0]
    assert (d["ctx_len"] - ctx).tolist() == [GAMMA + 1, 0, 3]
    assert d["anchor"].tolist() == [0, int(anchor[1]), 0] and step.n_committed.tolist() == [GAMMA + 1, 0, 3]
    assert (step.committed[1] == -1).all() and step.committed[2].tolist() == [0] * 3 + [-1] * (GAMMA - 2)


@pytest.mark.gpu
def test_refused_rows_do_not_carry_over(pkg):
    """A request whose parameters a later step refuses, or whose row it calls padding, takes nothing
    from the samples of the step before."""
    sizes = [20, 20, 20]
    d, rows = make(sizes, seed=5)
    d["row_parent"][:60] = torch.tensor([-1] + list(range(19)), dtype=torch.int32, device="cuda").repeat(3)
    d["row_tok"].zero_()
    d["logits"][:] = -1.0
    d["logits"][:, 0] = 50.0
    step = pkg.TreeStep(3, GAMMA, HQ, HKV, rows, 20)
    step.run(d)
    assert step.accept_len.tolist() == [GAMMA] * 3
    d["temperature"][1] = float("nan")
    d["row_req"][40 + 2] = -1
    ctx, anchor = d["ctx_len"].clone(), d["anchor"].clone()
    d["free_top"].fill_(d["free_pages"].numel())       # (pages enough: the caches are not read here)
    d["page_table"] = torch.nn.functional.pad(d["page_table"], (0, 2))
    step.run(d)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0x10
    assert step.accept_len.tolist() == [GAMMA, -1, 1] and step.row_sample[20:40].tolist() == [-1] * 20
    assert (d["ctx_len"] - ctx).tolist() == [GAMMA + 1, 0, 2] and int(d["anchor"][1]) == int(anchor[1])


@pytest.mark.gpu
def test_refused_distributions_do_not_carry_over(pkg):
    """VerifyStep from logits: the rows of a request that the sampler refuses have no distribution."""
    import harness
    wl = W.WORKLOADS["tiny"]
    d, step = harness.prepare(W.make_inputs(wl, seed=4), O.STATIC)
    rows = step.max_rows
    d["p_target"] = torch.full((rows, wl.vocab), 77.0, device="cuda")
    e = dict(d, logits=torch.randn(rows, wl.vocab, device="cuda"), temperature=torch.ones(wl.B, device="cuda"))
    e["temperature"][1] = float("nan")
    step.schedule(e, O.STATIC)
    step.pack(e, O.STATIC)
    step.distributions(e)
    assert pkg.read_device_error() == 0x10
    M = int(step.M_pack)
    p, req = d["p_target"], step.row_req[:M]
    assert (p[:M][req == 1] == 0).all() and (p[M:] == 77).all()
    assert ((p[:M][req != 1].sum(1) - 1).abs() < 1e-4).all()
