"""The verification step on the 4-bit cache, as a serving program runs it: schedule, pack,
norm and rotation of the projections at the packed positions, attention, acceptance and
the commit of the accepted rows, step after step; against the same calls made one by one
through the oracle on the kernel's own windows and acceptance."""
import math

import numpy as np
import pytest
import torch

import workloads as W
from oracle import dspark_oracle as O
from tests.test_verify_attn_kv4 import _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import speculative_decoding_verification_dspark_gb300 as p
    return p


@pytest.mark.parametrize("mode", [O.COMPACT, O.STATIC, O.CAP_ACCEPT])
def test_three_steps(pkg, mode):
    import harness
    wl = W.WORKLOADS["tiny"]
    inp = W.make_inputs(wl, seed=3)
    d = harness.device_inputs(inp)
    rows, Hq, Hkv = W.cap_rows(wl), wl.Hq, wl.Hkv
    gk, gv = 0.04, 0.03
    step = pkg.VerifyStep(wl.B, wl.gamma, Hq, Hkv, 128, 128, wl.vocab, rows, torch.float32, kv4=True)
    # the prompt's keys and values into the 4-bit cache
    n_pages, page = d["k_cache"].shape[0], d["k_cache"].shape[1]
    ctx0 = d["ctx_len"].cpu().numpy()
    cache = pkg.kv4_cache(n_pages, Hkv, page)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ctx0)]), dtype=torch.int32, device="cuda")
    flat = lambda c: torch.cat([  # noqa: E731
        c[d["page_table"][r].long()].flatten(0, 1)[:ctx0[r]] for r in range(wl.B)]).contiguous()
    pkg.kv4_store(flat(d.pop("k_cache")), flat(d.pop("v_cache")), cu,
                  torch.zeros(wl.B, dtype=torch.int32, device="cuda"), d["page_table"], cache, gk, gv)
    g = torch.Generator().manual_seed(5)
    wq, wk = (1 + 0.1 * torch.randn(128, generator=g) for _ in range(2))
    inv = (1e6 ** (-torch.arange(0, 128, 2) / 128)).float()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    d.update(kv_cache=cache, k_scale=gk, v_scale=gv, q_weight=wq.cuda(), k_weight=wk.cuda(),
             inv_freq=inv.cuda(), q=torch.zeros(rows, Hq, 128, **bf),
             k_new=torch.zeros(rows, Hkv, 128, **bf), v_new=torch.zeros(rows, Hkv, 128, **bf),
             p_target=torch.zeros(rows, wl.vocab, device="cuda"))
    for it in range(3):
        qkv = torch.randn(rows, (Hq + 2 * Hkv) * 128, generator=g).bfloat16().cuda()
        d["q_in"], d["k_in"], d["v_in"] = (x.unflatten(1, (-1, 128)) for x in qkv.split(
            [Hq * 128, Hkv * 128, Hkv * 128], 1))
        pt = torch.softmax(2 * torch.randn(rows, wl.vocab, generator=g), -1)
        d["p_target"].copy_(pt)
        before = {k: d[k].cpu().clone() for k in ("page_table", "ctx_len", "free_top", "kv_cache")}
        step.run(d, mode)
        torch.cuda.synchronize()
        assert pkg.read_device_error() == 0
        scu, M = step.cu_seqlens.cpu(), int(step.M_pack)
        pos = step.row_pos.cpu().numpy()
        pos[M:] = -1
        for name, wt, out in (("q_in", wq, "q"), ("k_in", wk, "k_new")):
            y, mag = O.qk_norm_rope(d[name].double().cpu().numpy(), wt.numpy(), 1e-6, inv.numpy(),
                                    False, 1.0, pos)
            err = np.abs(d[out].double().cpu().numpy() - y)[:M]
            assert np.all(err <= 2.0 ** -8 * np.abs(y[:M]) + 2.0 ** -18 * mag[:M])
        c = dict(q=d["q"].cpu(), k_new=d["k_new"].cpu(), v_new=d["v_new"].cpu(),
                 cache=before["kv_cache"], table=before["page_table"], cu=scu, gk=gk, gv=gv,
                 ctx=before["ctx_len"], hq=Hq, hkv=Hkv, page=page, M=M, scale=1.0 / math.sqrt(128))
        o, lse, to, tl = _reference(c)
        assert np.all(np.abs(step.out.double().cpu().numpy()[:M] - o) <= to)
        assert np.all(np.abs(step.lse.double().cpu().numpy()[:M] - lse) <= tl)
        acc = O.accept(pt.numpy(), d["p_draft"].cpu().numpy(), d["draft_tok"].cpu().numpy(),
                       d["uniforms"].cpu().numpy(), d["exp_noise"].cpu().numpy(),
                       step.windows.cpu().numpy(), scu.numpy(), mode, wl.gamma)
        keep = step.accept_len.cpu().numpy()
        assert np.array_equal(keep, acc.accept_len)
        ctx1 = d["ctx_len"].cpu().numpy()
        assert np.array_equal(ctx1, before["ctx_len"].numpy() + keep + 1)
        want = O.kv4_store(c["k_new"].float().numpy(), c["v_new"].float().numpy(), scu.numpy(),
                           before["ctx_len"].numpy(), d["page_table"].cpu().numpy(),
                           before["kv_cache"].numpy(), gk, gv, n_keep=keep + 1)
        assert np.array_equal(cache.cpu().numpy(), want)
    for refused in (lambda: step.graph(d, mode), lambda: step.pack_plan(d, mode),
                    lambda: step.attention_planned(d)):
        with pytest.raises(ValueError):
            refused()
