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


@pytest.mark.parametrize("D,bs,G,H", [(64, 8, 5, 3), (128, 16, 8, 2), (128, 32, 16, 1)])
@pytest.mark.parametrize("offset", [0.0, 4.0])
def test_codes_count_from_the_middle(D, bs, G, H, offset):
    """A weight's rounding counts with a code's distance from 7.5, not with the code: elements whose codes lie in
    the middle, and whose values are near zero, show it."""
    q, kc, vc, tables, lens = _problem([2, 3, 4, 5, 6, 7, 9, 12, 33] * 3, G * H, H, D, bs, seed=D + G,
                                       rows=lambda s, g: torch.randn(*s, generator=g) + offset)
    q = q.to(torch.bfloat16)
    want, bound, flat = exact.decode(q, kc, vc, tables, lens, D ** -0.5, bs)
    exact.check(_decode(q, kc, vc, tables, lens, D ** -0.5), want, bound, flat)


@pytest.mark.parametrize("qscale,scale", [(1.0, 3.0), (30.0, 0.088), (1.0, -0.7), (1e4, 0.088), (1e-3, 0.088)])
@pytest.mark.parametrize("vscale", [1.0, 1e-30, 1e30])
def test_sharp_and_flat_softmaxes(qscale, scale, vscale):
    """Logits from a few units to thousands: the bound narrows with the softmax."""
    D, bs, G, H = 128, 16, 4, 2
    q, kc, vc, tables, lens = _problem([1, 40, 333, 700], G * H, H, D, bs, seed=17,
                                       rows=lambda s, g: torch.randn(*s, generator=g) * vscale)
    q = (q * qscale).to(torch.bfloat16)
    want, bound, flat = exact.decode(q, kc, vc, tables, lens, scale, bs)
    # a flat softmax is near the plain average: only the sharp ones can be told from it
    exact.check(_decode(q, kc, vc, tables, lens, scale), want, bound, flat if qscale >= 1 else None, narrow=0.7)


def test_long_runs_do_not_drift():
    """220 stages of 32 tokens for every warp of the GPU.  The result rounded to bf16 differs from the 64-bit one's
    rounding only where the weights' fp16 rounding, 2^-11 / sqrt(12) * 1.2 = 1.7e-4 relative in the mean square for
    independent values, passes a border: sqrt(0.8 * 1.7e-4 * 2^-7.5) = 8.6e-4 in the mean square, half as much
    again allowed.  (An accumulator that only truncates loses 2^-24 of itself twice a stage: a drift of 2.6e-5 of
    the codes' sum, 2e-3 and more of these results, were it not kept near zero.)"""
    B, H, D, bs, L, pool = 16, 8, 128, 16, 131072, 512
    g = torch.Generator().manual_seed(5)
    caches = []
    for _ in range(2):
        b, p = ref.pack_row(*ref.quantise(torch.randn(pool, H, bs, D, generator=g).to(torch.bfloat16)))
        caches.append(torch.cat([b.flatten(2), p.flatten(2)], -1).contiguous())
    q = (torch.randn(B, H, D, generator=g) * 0.5).to(torch.bfloat16)
    tables = torch.stack([torch.cat([torch.randperm(pool, generator=g) for _ in range(L // bs // pool)])
                          for _ in range(B)]).to(torch.int32)
    got = _decode(q, *caches, tables, torch.full((B,), L, dtype=torch.int32), D ** -0.5)
    # every block comes equally often: the softmax is that over the pool
    k, v = (ref.values(c, bs, D).flatten(0, 1) for c in caches)
    p = torch.softmax(torch.einsum("bhd,thd->bht", q.double(), k) * D ** -0.5, -1)
    want = torch.einsum("bht,thd->bhd", p, v)
    off = (got - want.to(torch.bfloat16).double()).norm() / want.norm()
    assert float(off) <= 1.5 * 8.6e-4, float(off)


@pytest.mark.parametrize("ratio", [20, 26, 34, 60, 100])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("D,bs,G,H", [(128, 16, 8, 2), (64, 8, 12, 1)])
def test_value_row_far_above_the_others(D, bs, G, H, ratio, at):
    """A value row 2^ratio times the others, in sequences of one stage and of many.  It counts fully for a head that
    attends to it, and not at all for one whose weight for it is far below 2^-ratio."""
    lens = [20, 70, 700, 3000]
    q, kc, vc, tables, ln = _problem(lens, G * H, H, D, bs, seed=ratio)
    codes, pair = ref.quantise((torch.randn(len(lens), H, D, generator=torch.Generator().manual_seed(1))
                                * 2.0 ** ratio).to(torch.bfloat16))
    vb, vp = ref.pack_row(codes, pair)
    kb, kp = ref.pack_row(*ref.quantise(torch.full((H, D), 3.0).to(torch.bfloat16)))
    for i, n in enumerate(lens):
        t = {"first": 0, "middle": n // 2, "last": n - 1}[at]
        blk, o = int(tables[i, t // bs]), t % bs
        for cache, b, p in ((vc, vb[i], vp[i]), (kc, kb, kp)):
            cache[blk, :, o * D // 2:(o + 1) * D // 2] = b
            cache[blk, :, bs * D // 2 + 4 * o:bs * D // 2 + 4 * o + 4] = p
    # that row's key is 3 throughout: its logit is 3 scale sum q, far above or far below the others'
    q = q - q.mean(-1, keepdim=True)
    turn = torch.tensor([1.0 if h % 3 else -1.0 for h in range(G * H)])
    q = (q + turn[None, :, None] * 160.0 / (3.0 * D * D ** -0.5)).to(torch.bfloat16)
    want, bound, flat = exact.decode(q, kc, vc, tables, ln, D ** -0.5, bs)
    got = _decode(q, kc, vc, tables, ln, D ** -0.5)
    exact.check(got, want, bound)


def test_value_scales_at_random():
    """Value rows of all magnitudes from 2^-40 to 2^40, with logits that are as wide."""
    D, bs, G, H = 128, 16, 4, 3
    q, kc, vc, tables, lens = _problem([17, 90, 400, 900], G * H, H, D, bs, seed=3, rows=lambda s, g: torch.randn(
        *s, generator=g) * torch.exp2(torch.randint(-40, 41, (*s[:3], 1), generator=g).float()))
    q = (q * 12).to(torch.bfloat16)
    want, bound, _ = exact.decode(q, kc, vc, tables, lens, D ** -0.5, bs)
    exact.check(_decode(q, kc, vc, tables, lens, D ** -0.5), want, bound)


def test_scaled_row_of_no_weight_after_constant_rows():
    """Value rows of scale 0 set no range; a row of a large scale whose weight is 0 must leave the result alone."""
    D, bs, G, H, L = 128, 16, 4, 1, 200
    q, kc, vc, tables, lens = _problem([L, 40], G * H, H, D, bs, seed=2,
                                       rows=lambda s, g: torch.randn(*s[:3], 1, generator=g).expand(*s))
    vb, vp = ref.pack_row(*ref.quantise((torch.randn(1, D, generator=torch.Generator().manual_seed(1)) * 64).to(torch.bfloat16)))
    kb, kp = ref.pack_row(*ref.quantise(torch.full((1, D), 3.0).to(torch.bfloat16)))
    for i, t in ((0, 100), (0, 199), (1, 3)):
        blk, o = int(tables[i, t // bs]), t % bs
        for cache, b, p in ((vc, vb, vp), (kc, kb, kp)):
            cache[blk, :, o * D // 2:(o + 1) * D // 2] = b
            cache[blk, :, bs * D // 2 + 4 * o:bs * D // 2 + 4 * o + 4] = p
    q = q - q.mean(-1, keepdim=True)
    turn = torch.tensor([-1.0, 1.0, -1.0, -1.0])
    q = (q + turn[None, :, None] * 160.0 / (3.0 * D * D ** -0.5)).to(torch.bfloat16)
    want, bound, _ = exact.decode(q, kc, vc, tables, lens, D ** -0.5, bs)
    exact.check(_decode(q, kc, vc, tables, lens, D ** -0.5), want, bound)
