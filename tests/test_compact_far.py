"""Commits whose lengths come near 2^31, in the bf16 and the 4-bit cache: as at the same place of a
page near the start, and refused where the new length would pass 2^31 - 1."""
import pytest
import torch

PAGE, GAMMA = 1 << 20, 3


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import speculative_decoding_verification_dspark_gb300 as p
    return p


def commit(pkg, kv4, ctx, keep):
    """(error word, ctx_len after, the cache, n_committed) of a commit of `keep` rows at `ctx`, every
    page of the table being the same one."""
    dev = dict(device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, **dev)  # noqa: E731
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(GAMMA + 1, 1, 128, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.zeros(1, 2048, dtype=torch.int32, **dev)
    length, top, anchor = i32(ctx), i32(1), i32(7)
    com = torch.full((1, GAMMA + 1), -9, dtype=torch.int32, **dev)
    n = i32(-9)
    ws = torch.empty(pkg.compact_workspace_size(1), dtype=torch.uint8, **dev)
    head = (i32(0, GAMMA + 1), i32(keep - 1), i32(5), i32(*range(GAMMA))[None], table, length, anchor, i32(0), top)
    if kv4:
        cache = (pkg.kv4_cache(1, 1, PAGE),)
        cache[0].zero_()
        pkg.compact_kv4(k, v, *head, cache[0], com, n, ws)
    else:
        cache = tuple(torch.zeros(1, PAGE, 1, 128, dtype=torch.bfloat16, **dev) for _ in range(2))
        pkg.compact(k, v, *head, *cache, com, n, ws)
    torch.cuda.synchronize()
    return pkg.read_device_error(), int(length), cache, int(n)


@pytest.mark.gpu
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("end", [2 ** 31 - PAGE - 1, 2 ** 31 - PAGE, 2 ** 31 - PAGE + 3, 2 ** 31 - 1])
def test_commits_up_to_the_largest_length(pkg, kv4, end):
    for keep in (1, GAMMA + 1):
        err, length, cache, n = commit(pkg, kv4, end - keep, keep)
        assert (err, length, n) == (0, end, keep)
        at = (end - keep) % PAGE
        if at + keep > PAGE:                  # over a page's end: the one page holds both parts
            assert cache[0].any()
            continue
        want = commit(pkg, kv4, at, keep)[2]
        assert cache[0].any() and all(torch.equal(a, b) for a, b in zip(cache, want))


@pytest.mark.gpu
@pytest.mark.parametrize("kv4", [False, True])
def test_lengths_past_32_bits_are_refused(pkg, kv4):
    for ctx, keep in ((2 ** 31 - 1, 1), (2 ** 31 - GAMMA - 1, GAMMA + 1), (-1, 1), (-2 ** 31, 2)):
        err, length, cache, n = commit(pkg, kv4, ctx, keep)
        assert (err, length, n) == (0x10, ctx, -9)
        assert not any(c.any() for c in cache)
