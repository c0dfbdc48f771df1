"""GPU: the 4-bit decode within a bound counted token by token (_int4_exact.py)."""

import pytest
import torch

import _int4_exact as exact
import _int4_ref as ref
from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _problem(lens, Hq, H, D, bs, seed, rows=None):
    """Queries, caches of normal rows (or rows(shape, generator) for the values) and tables on the CPU."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    perm, at = torch.randperm(nb, generator=g).to(torch.int32), 0
    tables = torch.full((len(lens), max(1, max(need))), -5, dtype=torch.int32)
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    caches = []
    for make in (None, rows):
        x = torch.randn(nb, H, bs, D, generator=g) if make is None else make((nb, H, bs, D), g)
        b, p = ref.pack_row(*ref.quantise(x.to(torch.bfloat16)))
        caches.append(torch.cat([b.flatten(2), p.flatten(2)], -1).contiguous())
    q = torch.randn(len(lens), Hq, D, generator=g)
    return q, *caches, tables, torch.tensor(lens, dtype=torch.int32)


def _decode(q, kc, vc, tables, lens, scale):
    ws = ops.new_int4_workspace(q.shape[1], kc.shape[1], q.shape[2])
    out = ops.decode_int4(q.to(DEV), kc.to(DEV), vc.to(DEV), tables.to(DEV), lens.to(DEV), scale, ws)
    assert ops.device_status() == 0
    return out.cpu().double()


@pytest.mark.parametrize("D,bs,G,H", [(64, 16, 4, 2), (128, 16, 8, 2), (128, 8, 11, 1)])
@pytest.mark.parametrize("spread", [0, 6, 8, 10, 12])
def test_query_entries_far_apart(D, bs, G, H, spread):
    """One entry of each query head 2^spread times the others, which decide: it meets the same value in every key."""
    q, kc, vc, tables, lens = _problem([1, 40, 333, 700], G * H, H, D, bs, seed=D + spread)
    q[..., 5] = 2.0 ** spread
    q = q.to(torch.bfloat16)
    kc[:, :, :bs * D // 2].view(-1, H, bs, D // 2)[..., 2] &= 0x0F        # code 0 of dim 5
    pair = torch.tensor([0.375, -2.8125]).to(torch.bfloat16).view(torch.uint8)
    kc[:, :, bs * D // 2:] = pair.repeat(bs)
    want, bound, _ = exact.decode(q, kc, vc, tables, lens, D ** -0.5, bs, weight=2.0 ** -11, centre=0.0)
    exact.check(_decode(q, kc, vc, tables, lens, D ** -0.5), want, bound, narrow=0.85)
