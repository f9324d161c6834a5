"""The attention over the 4-bit cache shares its key tiles out among persistent CTAs.  Here single
tiles count: every group of tiles (request, KV head) has one heavy key in each tile at the edge of a
CTA's share and in its first and last tile, with a value of its own; all other keys weigh nothing.
A tile lost, taken twice or taken from another place then moves the result by 1 / (heavy keys)
of a value, and the lse by as much, against tolerances of 2^-8 and 2^-10 (checked too).

Tolerances: the heavy keys of a group have the same score s (all its terms equal and positive, sums
exact), so its weights are equal: the output is the mean of n values, off by the roundings of P to
fp16 (2^-11), of the sums over n <= 64 heavy keys (64 * 2^-23) and of the output to bf16 (2^-8 of the
value).  The other keys weigh e^-45 each, 2^21 of them 2^-43.  The lse is off by 136 * 2^-23 s, s < 26,
that is 2^-11.2, and the sums, 2^-17."""
import numpy as np
import pytest
import torch

from oracle import dspark_oracle as O
from tests.test_verify_attn_kv4 import pkg  # noqa: F401

pytestmark = pytest.mark.gpu
TILE = 128


def _blocks(n, hkv, gen):
    """n pages of 128 tokens with keys of -2 and values of random codes: light ones."""
    c = torch.randint(0, 256, (n, hkv, TILE // 16, O.KV4_BLOCK_BYTES), generator=gen, dtype=torch.uint8)
    c[..., :1024] = 0x66                                  # -2 in every element
    c[..., 2048:] = 0x38                                  # scales 1
    return c


# (per_sm: the CTAs of that query tile that share an SM)
@pytest.mark.parametrize("hint,per_sm", [(1, 4), (16, 3), (32, 2), (48, 2), (64, 2)])
@pytest.mark.parametrize("tiles", [16375, 16390])        # 64 groups: 2^20 - 576 and 2^20 + 384 in all
def test_each_tile_once(pkg, tiles, hint, per_sm):  # noqa: F811
    B, H = 8, 8
    gen = torch.Generator().manual_seed(tiles + hint)
    ctx = (tiles - 1) * TILE                              # and a tile of block rows
    ctas = pkg.load().dspark_num_sms() * per_sm
    U = B * H * tiles
    edges = {(c * U // ctas + d) for c in range(ctas + 1) for d in (-1, 0)}
    edges |= {g * tiles + d for g in range(B * H) for d in (0, tiles - 2)}
    heavy = {}                                            # (request, tile) -> its heads
    for u in edges:
        g, t = divmod(u, tiles)
        if 0 <= u < U and t < tiles - 1:
            heavy.setdefault((g // H, t), []).append(g % H)
    cache = _blocks(1 + len(heavy), H, gen)
    table = torch.zeros(B, tiles - 1, dtype=torch.int32)  # page 0 unless a tile has a heavy key
    tok = torch.randint(0, TILE, (len(heavy), H), generator=gen)
    for i, ((r, t), heads) in enumerate(heavy.items()):
        table[r, t] = 1 + i
        for h in heads:
            k = int(tok[i, h])
            cache[1 + i, h, k // 16, :1024].view(4, 16, 16)[:, k % 16] = 0xaa    # +2
    q = torch.ones(B, H, 128).bfloat16()
    q *= (1 + torch.arange(H) / 64)[None, :, None]
    kn = torch.full((B, H, 128), -2.0).bfloat16()
    vn = torch.randn(B, H, 128, generator=gen).bfloat16()
    d = [t.cuda() for t in (q, kn, vn, cache, table)]
    ctxd = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    out = torch.empty(B, H, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, H, device="cuda")
    ws = torch.empty(pkg.verify_attn_kv4_workspace_size(B, B, H, H, 32, hint), dtype=torch.uint8,
                     device="cuda")
    pkg.verify_attn_kv4(*d, ctxd, cu, 1 / np.sqrt(128), 32, out, lse, ws, max_block_rows=hint)
    torch.cuda.synchronize()
    assert pkg.read_device_error() == 0
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    pages = {k: 1 + i for i, k in enumerate(heavy)}
    for r in range(B):
        for h in range(H):
            at = [(p, int(tok[p - 1, h])) for k, p in pages.items() if k[0] == r and h in heavy[k]]
            blk = np.stack([cache[p, h, k // 16].numpy() for p, k in at])[:, None, None]
            v = O.kv4_values(blk, 1.0, 1.0)[1][np.arange(len(at)), [k % 16 for _, k in at], 0]
            n, s, mean = len(v), 256 * (1 + h / 64) / np.sqrt(128), v.mean(0)
            tol = 2.0 ** -8 * np.abs(mean) + (2.0 ** -11 + 2.0 ** -16) * np.abs(v).mean(0) + 1e-6
            assert 6 <= n <= 64
            for j in range(n):                            # any one of them would be missed
                assert np.any(np.abs(np.delete(v, j, 0).mean(0) - mean) > 2 * tol)
            assert np.log(n + 1) - np.log(n) > 2 * 2.0 ** -10
            assert np.all(np.abs(got[r, h] - mean) <= tol), (r, h, np.abs(got[r, h] - mean).max())
            assert abs(gl[r, h] - s - np.log(n)) <= 2.0 ** -10, (r, h, gl[r, h] - s - np.log(n))
