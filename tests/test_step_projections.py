"""The verification step from projections (q_in, k_in, v_in) on the bf16 cache: the same bits as
norm_rope called by hand and the step without them; the step graph, which has no norm, refuses."""
import pytest
import torch

import workloads as W
from oracle import dspark_oracle as O
from tests.test_kv4_cache import pkg  # noqa: F401


def test_graph_refuses_projections(pkg):  # noqa: F811
    step = pkg.VerifyStep(2, 4, 8, 2, 128, 128, 1024, 16, device="cpu")
    x = torch.zeros(16, 12 * 128, dtype=torch.bfloat16)
    q_in, k_in, v_in = (p.unflatten(1, (-1, 128)) for p in x.split([1024, 256, 256], 1))
    with pytest.raises(ValueError, match="norm_rope"):
        step.graph(dict(q_in=q_in, k_in=k_in, v_in=v_in), O.COMPACT)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [O.COMPACT, O.STATIC, O.CAP_ACCEPT])
def test_run_from_projections_on_the_bf16_cache(pkg, mode):  # noqa: F811
    import harness
    wl = W.WORKLOADS["tiny"]
    d, step = harness.prepare(W.make_inputs(wl, seed=4), mode)
    snap = harness.snapshot_state(d)
    rows, Hq, Hkv = step.max_rows, wl.Hq, wl.Hkv
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(rows, (Hq + 2 * Hkv) * 128, generator=g).bfloat16().cuda()
    parts = [x.unflatten(1, (-1, 128)) for x in qkv.split([Hq * 128, Hkv * 128, Hkv * 128], 1)]
    wq, wk = (1 + 0.1 * torch.randn(128, generator=g).cuda() for _ in range(2))
    inv = (1e6 ** (-torch.arange(0, 128, 2) / 128)).float().cuda()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    empty = lambda: [torch.zeros(rows, h, 128, **bf) for h in (Hq, Hkv, Hkv)]  # noqa: E731
    full = torch.zeros(rows, wl.vocab, dtype=d["p_target"].dtype, device="cuda")
    full[:d["p_target"].shape[0]] = d["p_target"]
    d["p_target"] = full
    d["q"], d["k_new"], d["v_new"] = empty()
    e = dict(d, q_in=parts[0], k_in=parts[1], v_in=parts[2], q_weight=wq, k_weight=wk, inv_freq=inv)
    step.run(e, mode)
    torch.cuda.synchronize()
    names = ("out", "lse", "accept_len", "out_tok", "committed", "n_committed")
    got = [getattr(step, n).clone() for n in names] + [d[k].clone() for k in ("k_cache", "v_cache")]
    rotated = [d[k].clone() for k in ("q", "k_new", "v_new")]
    M = int(step.M_pack)
    # by hand: the norm at the packed positions, then the step that reads q, k_new, v_new
    harness.restore_state(d, snap)
    d["q"], d["k_new"], d["v_new"] = empty()
    step.schedule(d, mode)
    step.pack(d, mode)
    pkg.qk_norm_rope(*parts, wq, wk, inv, step.row_pos, d["q"], d["k_new"], d["v_new"],
                     n_rows=step.M_pack)
    step.run(d, mode)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    for a, b in zip(rotated, (d["q"], d["k_new"], d["v_new"])):
        assert torch.equal(a, b) and bool(a[:M].any()) and not bool(a[M:].any())
    want = [getattr(step, n) for n in names] + [d["k_cache"], d["v_cache"]]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
