"""The 4-bit cache's factors k_scale and v_scale: refused outside 2^-100 .. 2^100, where a
derived factor (7 g, 16 g, 1 / (16 g), 3136 g, the attention's score factor) leaves fp32's normal
range; exact inside it."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O
from tests.test_kv4_cache import _case as _rows, pkg  # noqa: F401
from tests.test_verify_attn_kv4 import BOTH, _case, _check, _run

LO, HI = 2.0 ** -100, 2.0 ** 100
OUTSIDE = (np.nextafter(np.float32(LO), np.float32(0)), np.nextafter(np.float32(HI), np.float32(np.inf)),
           1e-45, 1.8e-40, 2.2e37, 5e37, 3.4e38)


def test_refused_outside(pkg):  # noqa: F811
    lib, f = pkg.load(), ctypes.c_void_p(4096)

    def calls(gk, gv, scale=0.1):
        return (lib.dspark_kv4_store(f, 256, f, 256, 1, f, f, 2, 8, 2, 16, f, 4, 9, gk, gv, f, None),
                lib.dspark_kv4_load(f, f, f, 2, 8, 2, 16, f, 4, 9, gk, gv, 1, f, f, None),
                lib.dspark_compact_kv4(f, f, 2, 8, f, f, f, f, 2, 4, 16, 4, 9, f, f, f, f, f, f, gk, gv,
                                       f, f, f, 1 << 20, None),
                attn(gk, gv, scale))

    def attn(gk, gv, scale):
        return lib.dspark_verify_attn_kv4(f, f, f, f, gk, gv, 9, f, 4, f, f, 2, 8, 8, 2, 16,
                                          ctypes.c_float(scale), 8, 4, f, f, f, 1 << 30, None)

    for g in OUTSIDE:
        assert calls(float(g), 1.0) == calls(1.0, float(g)) == (-1, -1, -1, -1), g
    for gk, scale in ((2.0 ** -100, 2.0 ** -40), (2.0 ** 100, 2.0 ** 30), (1.0, 1e-45), (1.0, 1e-39)):
        assert attn(gk, 1.0, scale) == -1, (gk, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("g", [LO, HI])
def test_store_and_load_at_the_ends(pkg, g):  # noqa: F811
    k, v, cu, p0, table, cache = _rows([20, 3], [5, 30], 2, 16, "f32", 7)
    k, v = k * g, v * g
    k[3, 0], v[4, 1, 5] = 1e38, float("inf")
    dev = cache.cuda()
    pkg.kv4_store(k.cuda(), v.cuda(), cu.cuda(), p0.cuda(), table.cuda(), dev, g, g)
    torch.cuda.synchronize()
    assert np.array_equal(dev.cpu().numpy(), O.kv4_store(k.numpy(), v.numpy(), cu.numpy(), p0.numpy(),
                                                         table.numpy(), cache.numpy(), g, g))
    ko, vo = (torch.empty(k.shape, device="cuda") for _ in range(2))
    pkg.kv4_load(dev, cu.cuda(), p0.cuda(), table.cuda(), ko, vo, g, g)
    for got, x in ((ko, k), (vo, v)):
        want = torch.tensor(O.kv4_quantise(x.numpy(), g)[2]).float()
        assert torch.equal(got.cpu(), want) and bool(want.isfinite().all())


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("gk,gv", [(LO, HI), (HI, LO)])
def test_attention_at_the_ends(pkg, hint, gk, gv):  # noqa: F811
    """Keys and values as large or small as their factors; the scale brings the scores back."""
    c = _case([300, 17], [4, 2], 8, 2, 16, seed=41, gk=gk, gv=gv, std=(16 * gk, 16 * gv))
    c["scale"] = float(np.float32(1 / (gk * 16 * np.sqrt(128))))
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    _check(c, out, lse)
