"""The 4-bit decode in 64 bits with a bound counted token by token, so that it
stays narrow for sharp softmaxes and for value rows far apart.

out = sum_t p_t v_t with p the softmax of x_t = scale (s_t Q_t + z_t sum q),
Q_t = sum_d q_d c_td.  To first order a relative error e_t of the weights moves
out by sum_t p_t e_t |v_t - out|, and e_t holds, in fp32 half steps h = 2^-24:
  * Q_t: D / 16 tensor core steps.  Each sums 16 products and the accumulator, cut
    25 bits below the largest exponent of theirs; a code is an fp16 subnormal, whose
    exponent counts as -14, so products of q_d c are cut at 2^-15 of the binade of the
    step's largest q_d (2^-19 where that is an odd dim's: those come as 16 c (q / 16)),
    each by less than that; the accumulator, 4 h of the magnitudes' sum,
  * sum q: D / 4 + 2 additions; z sum q, the multiply-add: 3 h of |z| sum |q| + |s Q|,
  * the logit times log2 e, from its maximum: 6 h of |x_t - max x|,
  * the exponential: 2^-22; every move of the running maximum, 32 tokens apart at
    most: 4 h of the weights before it.
The value product has sum_t p_t |s'_t| |c_td - centre| times `weight` (what a weight's
rounding to the tensor cores' operand is off by, codes being counted from `centre`),
weights below 2^-25 of the largest p_t s'_t an absolute 2^-35 of it; L / 16 steps, each
of which cuts its 16 products and the accumulator at 2^-15 of the largest of the 16
p_t |s'_t| (a product by no more than itself); the accumulator at 4 h of
sum_t p_t |s'_t| c_td, the zeros' part and the normaliser L / 8 + 16 additions at h, and
the output one rounding to bf16.
"""

from __future__ import annotations

import torch

import _int4_ref as ref

H32 = 2.0 ** -24


def _cut(aq, D):
    """What the tensor core steps of one head cut off sum_d |q_d| c_d: [..., D] -> [...].  Lane c of four holds dims
    c D / 4 on, in words of 8; a step takes dims 0, 4 (even) and 1, 5 (odd) of a word of each, or 2, 6 and 3, 7."""
    q = aq.unflatten(-1, (4, D // 32, 8))
    total = 0
    for even, odd in (((0, 4), (1, 5)), ((2, 6), (3, 7))):
        unit = torch.maximum(q[..., even].amax((-1, -3)), q[..., odd].amax((-1, -3)) / 16) * 2.0 ** -15   # [..., words]
        total = total + 17 * unit.sum(-1)
    return total


def decode(query, key_cache, value_cache, tables, lens, scale, block_size, *, weight=2.0 ** -11, centre=7.5):
    """(out, bound, uniform) fp64 [B, Hq, D]; uniform: the plain average of the values."""
    B, Hq, D = query.shape
    bs = block_size
    scale = float(torch.tensor(scale, dtype=torch.float32))
    k, v = ref.values(key_cache, bs, D), ref.values(value_cache, bs, D)
    ks, kz = ref.pairs(key_cache, bs, D)
    vs, vz = ref.pairs(value_cache, bs, D)
    H = k.shape[2]
    G = Hq // H
    out, bound, flat = (torch.zeros(B, H, G, D, dtype=torch.float64) for _ in range(3))
    for i in range(B):
        L = min(int(lens[i]), tables.shape[1] * bs)
        if L <= 0:
            continue
        ids = tables[i, :-(-L // bs)].long()
        row = lambda t: t[ids].flatten(0, 1)[:L]  # noqa: E731
        kk, vv = row(k), row(v)                                    # [L, H, D]
        s, z, s2, z2 = (row(t) for t in (ks, kz, vs, vz))          # [L, H]
        kc = torch.where(s[..., None] != 0, (kk - z[..., None]) / s[..., None], 0.0).round()
        vc = torch.where(s2[..., None] != 0, (vv - z2[..., None]) / s2[..., None], 0.0).round()
        q = query[i].double().view(H, G, D)
        x = torch.einsum("hgd,thd->hgt", q, kk) * scale
        p = torch.softmax(x, -1)
        o = torch.einsum("hgt,thd->hgd", p, vv)
        aq = q.abs()
        sq = s.abs().t()[:, None] * torch.einsum("hgd,thd->hgt", aq, kc)          # [H, G, L]: |s| sum |q| c
        zq = z.abs().t()[:, None] * aq.sum(-1, keepdim=True)
        dx = abs(scale) * (H32 * ((D / 4 + 8) * zq + (D / 4 + 4) * sq) + s.abs().t()[:, None] * _cut(aq, D)[..., None])
        e = dx + 6 * H32 * (x.amax(-1, keepdim=True) - x) + 2.0 ** -22 + (L / 32 + 2) * 4 * H32
        far = torch.stack([(vv[:, h][None] - o[h][:, None]).abs() for h in range(H)])  # [H, G, L, D]
        b = torch.einsum("hgt,hgtd->hgd", p * e, far) * (1 + 4 * float((p * e).sum(-1).max()))
        w = p * s2.abs().t()[:, None]                                              # [H, G, L]
        b += weight * torch.einsum("hgt,thd->hgd", w, (vc - centre).abs())
        b += (L * 15 * 2.0 ** -34) * w.amax(-1, keepdim=True)
        tiles = torch.nn.functional.pad(w, (0, -L % 16)).unflatten(-1, (-1, 16))   # [H, G, tiles, 16]
        unit = tiles.amax(-1, keepdim=True) * 2.0 ** -15
        b += (torch.minimum(15 * tiles, unit).sum((-1, -2)) + unit.sum((-1, -2)))[..., None]
        b += (L / 16 + 4) * 4 * H32 * (torch.einsum("hgt,thd->hgd", w, vc) + centre * w.sum(-1, keepdim=True))
        zc = (z2 + centre * s2).abs() + z2.abs()
        b += (L / 8 + 16) * H32 * (torch.einsum("hgt,th->hg", p, zc)[..., None] + o.abs())
        out[i], bound[i] = o, 1.01 * b + ref.half_step(torch.bfloat16) * 1.01 * o.abs() + 2.0 ** -134
        flat[i] = vv.mean(0)[:, None].expand(H, G, D)
    return tuple(t.reshape(B, Hq, D) for t in (out, bound, flat))


def check(got, want, bound, flat=None, narrow=0.9):
    """The result lies within the bound, and the bound tells it from zeros (and from the plain average, where given)
    in at least the share `narrow` of the elements of sequences that have tokens."""
    live = (want.abs().amax((1, 2)) > 0)
    err = (got - want).abs()
    assert bool((err <= bound).all()), \
        f"worst {float((err / bound).max()):.3f} of the bound, {int((err > bound).sum())} elements"
    if bool(live.any()) and narrow:
        assert float((want.abs() > bound)[live].double().mean()) >= narrow, "zeros would pass"
        if flat is not None:
            assert float(((flat - want).abs() > bound)[live].double().mean()) >= narrow, "a plain average would pass"
