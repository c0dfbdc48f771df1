"""GPU: the 4-bit decode over the longest sequence that a table row holds, 2^31 - 11 tokens."""

import pytest
import torch

import _int4_exact as exact
import _int4_ref as ref
from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_longest_sequence():
    """2^28 - 1 blocks of 8 tokens: 63 of them in turn, and at the end one that outweighs them all, with 5 of its
    rows within the length and NaN in the other 3."""
    D, bs, pool = 64, 8, 64
    blocks, L = 2 ** 28 - 1, 2 ** 31 - 11
    g = torch.Generator().manual_seed(1)
    k = torch.randn(pool, 1, bs, D, generator=g) * 0.1
    v = torch.randn(pool, 1, bs, D, generator=g)
    k[-1] = 3 + 0.1 * k[-1]
    caches = []
    for x in (k, v):
        b, p = ref.pack_row(*ref.quantise(x.to(torch.bfloat16)))
        caches.append(torch.cat([b.flatten(2), p.flatten(2)], -1).contiguous())
    q = torch.full((1, 2, D), 1.0) + 0.5 * torch.randn(1, 2, D, generator=g)
    q = q.to(torch.bfloat16)
    # the last block's logits stand some 190 above the others': they outweigh 2^31 of them
    want, bound, flat = exact.decode(q, *caches, torch.tensor([[pool - 1]], dtype=torch.int32),
                                     torch.tensor([5], dtype=torch.int32), 1.0, bs)
    dev = [c.to(DEV) for c in caches]
    for c in dev:
        c[-1, :, bs * D // 2 + 4 * 5:] = 0xFF
    tables = (torch.arange(blocks, device=DEV) % (pool - 1)).to(torch.int32)[None].contiguous()
    tables[0, -1] = pool - 1
    lens = torch.tensor([L], dtype=torch.int32, device=DEV)
    ws = ops.new_int4_workspace(2, 1, D)
    out = ops.decode_int4(q.to(DEV), *dev, tables, lens, 1.0, ws)
    exact.check(out.cpu().double(), want, bound, flat)
    # and a sum over all of them: every block's rows as often as it comes
    lens.fill_(L - 5)
    out = ops.decode_int4(q.to(DEV) * 0.125, *dev, tables, lens, 1.0, ws).cpu().double()
    kk, vv = (ref.values(c[:-1], bs, D).flatten(0, 1)[:, 0] for c in caches)
    times = torch.full((pool - 1,), (blocks - 1) // (pool - 1), dtype=torch.float64)
    times[:(blocks - 1) % (pool - 1)] += 1
    p = torch.softmax((q[0].double() * 0.125) @ kk.t() + times.repeat_interleave(bs).log(), -1)
    full = p @ vv
    # Each warp of 148 x 4 x 4 adds up 2^26 / 2368 = 28341 stages in fp32: that many half steps of 2^-24 for the
    # normaliser and for the zeros' part, 4 half steps (truncation) twice a stage for the codes' part (magnitudes
    # below 7.5 + 15 scales), the weights' rounding on top: no narrower proof for so many, 2 to 3 % of a value
    s2, z2 = (t[:, :, 0].flatten() for t in ref.pairs(caches[1][:-1], bs, D))
    n, h = 28341, 2.0 ** -24
    sums = n * h * (p @ (z2 + 7.5 * s2).abs())[:, None] + n * h * full.abs() + 8 * n * h * (p @ (22.5 * s2))[:, None]
    weights = 2.0 ** -11 * torch.einsum("ht,t,td->hd", p, s2, ((vv - z2[:, None]) / s2[:, None] - 7.5).abs())
    assert bool(((out[0] - full).abs() <= sums + weights + 2.0 ** -8 * 1.01 * full.abs()).all())
    assert ops.device_status() == 0
