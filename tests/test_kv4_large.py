"""The norm with rotation and the 4-bit cache's calls where offsets pass 2^31 elements and 2^32
bytes, and on batches without a row."""
import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O
from tests.test_kv4_cache import _case as _rows, pkg  # noqa: F401
from tests.test_qk_norm_rope import _check as _check_rope, _inputs, _outputs
from tests.test_verify_attn_kv4 import BOTH, _case, _check, _run

pytestmark = pytest.mark.gpu
PAGE_BYTES = 8 * O.KV4_BLOCK_BYTES                      # 16 tokens of 8 heads
FAR = 260000                                            # pages, 4.5 GB
PLACES = [2 ** 31 // PAGE_BYTES, 2 ** 31 // PAGE_BYTES + 1, 2 ** 32 // PAGE_BYTES,
          2 ** 32 // PAGE_BYTES + 1, FAR - 1, 0]


def _far(rows):
    """bf16 / fp32 rows a gigaelement apart: the third begins at element 2^31."""
    buf = torch.empty(2 ** 31 + rows[0].numel(), dtype=rows.dtype, device="cuda")
    view = buf.as_strided(rows.shape, (2 ** 30, 128, 1))
    view.copy_(rows)
    return view


def test_pages_and_rows_far_out(pkg):  # noqa: F811
    k, v, cu, p0, table, small = _rows([3], [77], 8, 16, "bf16", 1)   # 80 positions: 5 pages
    n = table.shape[1]
    far = torch.tensor([PLACES[:n]], dtype=torch.int32)
    cache = torch.empty(FAR, 8, 1, O.KV4_BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    for i in range(n):
        cache[PLACES[i]] = small[int(table[0, i])].cuda()
    pkg.kv4_store(_far(k), _far(v), cu.cuda(), p0.cuda(), far.cuda(), cache, 0.25, 0.5)
    ko, vo = (torch.empty(3, 8, 128, device="cuda") for _ in range(2))
    pkg.kv4_load(cache, cu.cuda(), p0.cuda(), far.cuda(), ko, vo, 0.25, 0.5)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    want = O.kv4_store(k.float().numpy(), v.float().numpy(), cu.numpy(), p0.numpy(), table.numpy(),
                       small.numpy(), 0.25, 0.5)
    for i in range(n):
        assert np.array_equal(cache[PLACES[i]].cpu().numpy(), want[int(table[0, i])])
    for got, x, g in ((ko, k, 0.25), (vo, v, 0.5)):
        assert torch.equal(got.cpu(), torch.tensor(O.kv4_quantise(x.float().numpy(), g)[2]).float())


@BOTH
def test_attention_far_out(pkg, hint):  # noqa: F811
    """The last two rows of q and out of 4.5 GB each, over pages of a 4.5 GB cache."""
    c = _case([93], [2], 16, 8, 16, seed=51)
    rows, n = 1100000, c["table"].shape[1]
    big = dict(c, M=rows, cu=torch.tensor([rows - 2, rows], dtype=torch.int32),
               table=torch.tensor([PLACES[:n]], dtype=torch.int32))
    assert n <= len(PLACES)
    cache = torch.empty(FAR, 8, 1, O.KV4_BLOCK_BYTES, dtype=torch.uint8, device="cuda")
    for i in range(n):
        cache[PLACES[i]] = c["cache"][int(c["table"][0, i])].cuda()
    big["cache"] = cache
    for name in ("q", "k_new", "v_new"):
        big[name] = torch.empty(rows, *c[name].shape[1:], dtype=torch.bfloat16, device="cuda")
        big[name][-2:] = c[name].cuda()
    call, out, lse = _run(pkg, big, hint)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    assert bool((out[:-2] == 5.0).all()) and bool((lse[:-2] == 5.0).all())
    _check(c, out[-2:], lse[-2:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_of_rows_far_apart(pkg, dtype):  # noqa: F811
    parts, dev, pos, w, inv = _inputs(3, 0, 8, 2, 128, dtype, False, True, 5000)
    outs = _outputs(3, 8, 2)
    far = [_far(p) for p in dev]
    pkg.qk_norm_rope(*far, *[t.cuda() for t in w], inv.cuda(), pos.cuda(), *outs)
    torch.cuda.synchronize()
    _check_rope(parts, outs, pos, w, inv, False, 1.0, 1e-6)


def test_batches_without_a_row(pkg):  # noqa: F811
    """Requests without rows, and rows that no request has: nothing is written."""
    for hint in (1, 4, 16):
        c = _case([20, 40], [0, 0], 8, 2, 16, seed=52, tail=5)
        call, out, lse = _run(pkg, c, hint)
        call()
        assert pkg.read_device_error() == 0
        assert bool((out == 5.0).all()) and bool((lse == 5.0).all())
    cache, cu, p0 = c["cache"].cuda(), c["cu"].cuda(), c["ctx"].cuda()
    before, table = cache.clone(), c["table"].cuda()
    k = torch.full((5, 2, 128), float("nan"), device="cuda")
    pkg.kv4_store(k, k, cu, p0, table, cache, 1.0, 1.0)
    ko = torch.full((5, 2, 128), 9.0, device="cuda")
    pkg.kv4_load(cache, cu, p0, table, ko, ko.clone(), 1.0, 1.0)
    assert pkg.read_device_error() == 0
    assert torch.equal(cache, before) and bool((ko == 9.0).all())
    _, dev, pos, w, inv = _inputs(5, 0, 8, 2, 128, "bf16", False, True, 50)
    for n in (0, -3):
        outs = _outputs(5, 8, 2)
        pkg.qk_norm_rope(*dev, *[t.cuda() for t in w], inv.cuda(), pos.cuda(), *outs,
                         n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert all(bool((o == 7.0).all()) for o in outs)
    assert pkg.read_device_error() == 0
