"""GPU: the 4-bit decode over value scales that the store never writes or that lie far apart."""

import pytest
import torch

import _int4_ref as ref
from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _cache(codes, pair):
    """CPU cache [nb, H, record] of codes [nb, H, bs, D] and (scale, zero) pairs [nb, H, bs, 2]."""
    b, p = ref.pack_row(codes, pair.to(torch.bfloat16))
    return torch.cat([b.flatten(2), p.flatten(2)], -1).contiguous()


def _normal_cache(nb, H, bs, D, g):
    return _cache(*ref.quantise(torch.randn(nb, H, bs, D, generator=g).to(torch.bfloat16)))


def _decode(q, kc, vc, tables, lens, scale):
    ws = ops.new_int4_workspace(q.shape[1], kc.shape[1], q.shape[2])
    out = ops.decode_int4(q.to(DEV), kc.to(DEV), vc.to(DEV), tables.to(DEV), lens.to(DEV), scale, ws)
    assert ops.device_status() == 0
    return out.cpu().double()


@pytest.mark.parametrize("D,bs,G,H", [(64, 8, 3, 2), (128, 16, 4, 2), (128, 32, 12, 1)])
@pytest.mark.parametrize("which", ["values", "mixed values", "keys"])
def test_negative_scales(D, bs, G, H, which):
    """zero + scale c counted from the other end: 15 - c, -scale and zero + 15 scale, all exact here."""
    lens = torch.tensor([1, 40, 333, 0, 700], dtype=torch.int32)
    width = -(-700 // bs)
    nb = 5 * width
    g = torch.Generator().manual_seed(D + bs)
    tables = torch.randperm(nb, generator=g).to(torch.int32).view(5, width)
    q = torch.randn(5, G * H, D, generator=g).to(torch.bfloat16)
    codes = torch.randint(0, 16, (nb, H, bs, D), generator=g, dtype=torch.uint8)
    scale = torch.exp2(torch.randint(-3, 2, (nb, H, bs, 1), generator=g).float())
    turned = torch.rand(nb, H, bs, 1, generator=g) < (0.5 if which == "mixed values" else 2.0)
    plain = _cache(codes, torch.cat([scale, -7.5 * scale], -1))
    other = _cache(torch.where(turned, 15 - codes, codes),
                   torch.cat([torch.where(turned, -scale, scale), torch.where(turned, 7.5 * scale, -7.5 * scale)], -1))
    assert torch.equal(ref.values(plain, bs, D), ref.values(other, bs, D))
    rest = _normal_cache(nb, H, bs, D, g)
    a, b = ((plain, rest), (other, rest)) if which == "keys" else ((rest, plain), (rest, other))
    want, bound = ref.decode(q, *a, tables, lens, 0.1, bs)
    got = _decode(q, *b, tables, lens, 0.1)
    assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
