"""Verify attention over the 4-bit cache: values that are not numbers in block rows that some
of the query rows do not see, and pages out of range.  Reference and tolerances are those of test_verify_attn_kv4."""
import pytest
import torch

from tests.test_verify_attn_kv4 import BOTH, _case, _check, _reference, _run, pkg  # noqa: F401

NAN = float("nan")


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("ctx,lens,page", [([200, 40], [5, 2], 16), ([0, 5], [9, 1], 16),
                                           ([5000, 130], [4, 150], 64), ([90], [300], 32)])
def test_nan_in_a_block_rows_value(pkg, hint, ctx, lens, page):  # noqa: F811
    """A NaN in v_new reaches the rows from its own on, in its channel and its heads; the rows
    before it, which do not see it, and every other channel are as ever."""
    c = _case(ctx, lens, 8, 2, page, seed=21)
    cu, at = c["cu"].tolist(), []      # (first row, last row + 1, KV head, channel)
    for r, n in enumerate(lens):
        for row, h, ch in ((n // 2, 1, 7), (n - 1, 1, 7), (n - 1, 0, 64), (n // 3, 0, 127), (0, 1, 96)):
            at.append((cu[r] + row, cu[r + 1], h, ch))
            c["v_new"][cu[r] + row, h, ch] = NAN
    call, out, lse = _run(pkg, c, hint, 32)
    call()
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    c["v_new"] = torch.nan_to_num(c["v_new"], nan=0.0)
    o = torch.tensor(_reference(c)[0])
    seen = torch.zeros(out.shape, dtype=torch.bool)
    for a, z, h, ch in at:
        seen[a:z, 4 * h:4 * h + 4, ch] = True
    got = out.cpu()
    assert torch.equal(got.isnan(), seen)
    _check(c, torch.where(seen, o.to(torch.bfloat16), got), lse)


@pytest.mark.gpu
@BOTH
def test_nan_in_a_block_rows_key(pkg, hint):  # noqa: F811
    """A NaN in k_new makes the rows that see it NaN, and no others."""
    c = _case([200, 40], [5, 2], 8, 2, 16, seed=22)
    c["k_new"][3, 1, 5] = NAN
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    c["k_new"][3, 1, 5] = 0
    o, l, _, _ = _reference(c)
    assert bool(out[3:5, 4:].isnan().all()) and bool(lse[3:5, 4:].isnan().all())
    out[3:5, 4:] = torch.tensor(o[3:5, 4:]).bfloat16().cuda()
    lse[3:5, 4:] = torch.tensor(l[3:5, 4:]).float().cuda()
    _check(c, out, lse)


@pytest.mark.gpu
@BOTH
def test_infinite_values_in_unseen_rows(pkg, hint):  # noqa: F811
    c = _case([200, 40], [5, 2], 8, 2, 16, seed=23)
    keep = c["v_new"][4].clone()
    c["v_new"][4, :, ::3], c["k_new"][4, 0, 1] = float("inf"), -float("inf")
    call, out, lse = _run(pkg, c, hint)
    call()
    torch.cuda.synchronize()
    c["v_new"][4], c["k_new"][4, 0, 1] = keep, 0
    o, l, _, _ = _reference(c)         # (row 4 itself sees them)
    out[4], lse[4] = torch.tensor(o[4]).bfloat16().cuda(), torch.tensor(l[4]).float().cuda()
    _check(c, out, lse)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("page", [-1, -2 ** 31 + 1, -2 ** 31, 2 ** 31 - 1])
def test_every_page_out_of_range_is_reported(pkg, hint, page):  # noqa: F811
    c = _case([200, 100], [3, 2], 8, 2, 16, seed=24)
    c["table"][0, 12] = page
    call, out, lse = _run(pkg, c, hint)
    call()
    assert pkg.read_device_error() == 0x10
    c["table"][0, 12] = 0              # (the other request is as ever)
    o, l, _, _ = _reference(c)
    out[:3], lse[:3] = torch.tensor(o[:3]).bfloat16().cuda(), torch.tensor(l[:3]).float().cuda()
    _check(c, out, lse)
